"""Corners of the layer's operators: gates below the normal range, rows with NaN, temporaries of a call on another
stream, host tensors at the raw entry points, and other calls that the documentation allows or has to refuse.

Tolerances are those of test_recurrence.py and test_qk_norm.py, counted in roundings there."""
import pytest
import torch

from tests import _layer_ref as ref
from tests._util import BF16_TOL


# ------------------------------------------------------------------ CPU: what a call allocates on which stream

def _fake_calls(pk, monkeypatch):
    """The package's calls with the library, the streams and the norms replaced by fakes: a list of
    (call, name, whether it was allocated on the call's stream) for every tensor that reaches the library."""
    import contextlib
    inside, where, seen = [0], {}, []

    @contextlib.contextmanager
    def stream(s):
        inside[0] += 1
        yield
        inside[0] -= 1

    def made(f):
        def make(*a, **kw):
            kw.pop("device", None), kw.pop("pin_memory", None)
            t = f(*a, **kw)
            where[id(t)] = (inside[0] > 0, t)
            return t
        return make

    def raw(call, names):
        def fake(p, *args):
            seen.extend((call, n, where[id(t)][0]) for n, t in zip(names, args) if id(t) in where)
        return fake

    monkeypatch.setattr(pk.torch.cuda, "stream", stream)
    monkeypatch.setattr(pk.torch, "empty", made(torch.empty))
    monkeypatch.setattr(pk.torch, "empty_like", made(torch.empty_like))
    for n in ("osdn_fwd_workspace_size", "osdn_bwd_workspace_size"):
        monkeypatch.setattr(pk, n, lambda p: 256)
    monkeypatch.setattr(pk, "osdn_fwd_host_buffer_size", lambda p, groups: 256)
    fwd = "q k v beta r d0 S0 out final_S final_d workspace".split()
    bwd = "q k v beta r d0 S0 dout dS_final dd_final dq dk dv dbeta dr dd0 dS0 workspace".split()
    monkeypatch.setattr(pk, "osdn_fwd", raw("forward", fwd))
    monkeypatch.setattr(pk, "osdn_fwd_host", raw("forward_host", fwd))
    monkeypatch.setattr(pk, "osdn_bwd", raw("backward", bwd))
    monkeypatch.setattr(pk, "osdn_fwd_scan_diag", raw("residual_ratio", "k beta r d0 d rho q_geo workspace".split()))
    return seen


class _FakeNorm:
    def apply(self, q, k, positions=None, stream=None):
        return q.clone(), k.clone()

    def gradients(self, q, k, dq, dk, positions=None, stream=None):
        return {"dq": dq.clone(), "dk": dk.clone(), "dwq": None, "dwk": None}


def test_what_a_call_drops_is_allocated_on_its_stream(monkeypatch):
    """Workspaces, and with qk the gradients of the normalised q and k, are dropped when the call returns, with its
    kernels still ahead: they have to come from the pool of the stream that these run on."""
    import preconditioned_delta_rule_token_b200 as pk
    seen = _fake_calls(pk, monkeypatch)
    q, b, s = torch.zeros(1, 4, 1, 64), torch.zeros(1, 4, 1), object()
    pk.forward(q, q, q, b, stream=s, qk=_FakeNorm())
    pk.backward(q, q, q, b, q, stream=s, qk=_FakeNorm())
    pk.residual_ratio(q, b, stream=s)
    pk.forward_host(q, q, q, b, stream=s)
    dropped = [e for e in seen if e[1] == "workspace" or e[:2] in (("backward", "dq"), ("backward", "dk"))]
    assert len(dropped) == 6 and all(e[2] for e in dropped), dropped
    kept = [e for e in seen if e not in dropped]
    assert kept and not any(e[2] for e in kept)      # results: on the caller's stream, as without qk



@pytest.mark.parametrize("heads", ((4, 2), (2, 4)))
def test_the_delta_rule_wants_as_many_key_heads(monkeypatch, heads):
    """qk_norm takes shared key heads, forward, backward and step do not: they refuse them before any kernel."""
    import preconditioned_delta_rule_token_b200 as pk
    seen = _fake_calls(pk, monkeypatch)
    (q, k), b = (torch.zeros(1, 4, n, 64) for n in heads), torch.zeros(1, 4, heads[1])
    v, S, d = torch.zeros_like(k), torch.zeros(1, heads[1], 64, 64), torch.zeros(1, heads[1], 64)
    for call in (lambda: pk.forward(q, k, v, b, qk=_FakeNorm()), lambda: pk.backward(q, k, v, b, v, qk=_FakeNorm()),
                 lambda: pk.step(q[:, 0], k[:, 0], v[:, 0], b[:, 0], S, d, qk=_FakeNorm())):
        with pytest.raises(pk.OsdnError, match="one shape"):
            call()
    assert not seen


_RAW = {
    "osdn_recur_fwd": "x gate h0 lengths h final_h checkpoints",
    "osdn_recur_bwd": "x gate h0 lengths dh dfinal_h checkpoints dx dgate dh0 workspace",
    "osdn_recur_step": "x gate state h",
    "osdn_qk_fwd": "q k wq wk positions freqs lengths q_out k_out",
    "osdn_qk_bwd": "q k wq wk positions freqs lengths dq_out dk_out dq dk dwq dwk workspace",
    "osdn_rope": "x positions freqs lengths out",
}


class _Fake(torch.Tensor):
    """A host tensor that says it is on a CUDA device (its address never reaches the library here)."""
    @property
    def is_cuda(self):
        return True


@pytest.mark.parametrize("call,name", [(c, n) for c, names in _RAW.items() for n in names.split()])
def test_raw_calls_refuse_host_and_strided_tensors(osdn_lib, monkeypatch, call, name):
    """Every tensor argument: a host tensor, and one whose last dimension is not contiguous, is refused before the
    library sees an address; optional ones may be None."""
    import preconditioned_delta_rule_token_b200 as pk
    reached = []

    class Library:
        def __getattr__(self, n):
            return lambda *a: reached.append(n) or 0

    monkeypatch.setattr(osdn_lib, "lib", Library)
    monkeypatch.setattr(osdn_lib, "_handle", lambda stream: 0)
    names = _RAW[call].split()
    good = lambda: torch.zeros(4, 6).as_subclass(_Fake)  # noqa: E731
    getattr(pk, call)(None, *[good() for _ in names])
    assert reached == [call]
    for bad in (torch.zeros(4, 6), torch.zeros(6, 4).as_subclass(_Fake).t()):
        with pytest.raises(pk.OsdnError):
            getattr(pk, call)(None, *[bad if n == name else good() for n in names])
    getattr(pk, call)(None, *[None if n == name else good() for n in names])   # NULL: the library's own check
    assert reached == [call, call]



class _FakeCalls:
    """The extension module's functions on fake tensors; `reached` lists the library's functions called."""
    def __init__(self):
        self.reached = []

    def layouts(self, *ts):
        return repr([None if t is None else (t.dtype, t.shape, t.stride()) for t in ts])

    def here(self, t):
        return True

    def like(self, t):
        return torch.empty(t.shape, dtype=t.dtype)

    def floats(self, t, *sizes):
        return torch.empty(sizes)

    def __getattr__(self, name):
        return lambda params, *a: self.reached.append((name, params, a)) or 0


@pytest.fixture
def fake_layer(monkeypatch):
    """The layer's wrappers without a GPU: (module, its calls)."""
    from preconditioned_delta_rule_token_b200 import _layer
    calls = _FakeCalls()
    monkeypatch.setattr(_layer, "_C", calls)
    monkeypatch.setattr(_layer, "_RECUR", _layer._Kept())
    monkeypatch.setattr(_layer, "_HEADS", _layer._Kept())
    return _layer, calls


def _fake(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Fake)


def test_given_workspaces_are_checked(fake_layer):
    """A workspace on the host, not dense (its elements are more than its memory) or no tensor is refused before the
    call."""
    import preconditioned_delta_rule_token_b200 as pk
    layer, calls = fake_layer
    x, q, w = _fake(2, 100, 16), _fake(2, 5, 1, 64), _fake(64)
    for call, name in ((lambda ws: layer.recurrence_backward(x, x, x, workspace=ws), "recur_bwd"),
                       (lambda ws: layer.qk_norm_backward(q, q, q, q, wq=w, workspace=ws), "qk_bwd")):
        for ws in (torch.zeros(1 << 20), _fake(1).expand(1 << 20), _fake(64, 64).t(), 1 << 20):
            with pytest.raises(pk.OsdnError):
                call(ws)
        assert not calls.reached
        call(_fake(1 << 10))
        assert calls.reached.pop()[0] == name


def test_numbers_are_taken_by_value(fake_layer):
    """A scale, an eps or an amplitude held in a tensor that changes in place between two calls: each call has the
    value of its time. What is no number is refused."""
    import preconditioned_delta_rule_token_b200 as pk
    layer, calls = fake_layer
    q, f = _fake(2, 5, 1, 64), _fake(32, dtype=torch.float64)
    field = {"scale": "scale_q"}

    def params(call):
        call()
        address = calls.reached[-1][1]
        return layer.B.osdn_qk_params.from_address(address)

    for name, call in [(n, lambda **kw: layer.qk_norm(q, q, f, **kw)) for n in ("eps", "amplitude", "scale_q", "scale_k")] + \
                      [(n, lambda **kw: layer.qk_norm_backward(q, q, q, q, f, **kw)) for n in ("eps", "scale_k")] + \
                      [(n, lambda **kw: layer.rope(q, f, **kw)) for n in ("amplitude", "scale")]:
        t = torch.tensor(0.5)
        assert getattr(params(lambda: call(**{name: t})), field.get(name, name)) == 0.5
        t.fill_(2.0)
        assert getattr(params(lambda: call(**{name: t})), field.get(name, name)) == 2.0
        for bad in ("x", torch.ones(2), None):
            with pytest.raises(pk.OsdnError):
                call(**{name: bad})
    p = torch.tensor(3)
    assert params(lambda: layer.rope(q, f, pos0=p)).pos0 == 3
    p += 1
    assert params(lambda: layer.rope(q, f, pos0=p)).pos0 == 4
    with pytest.raises(pk.OsdnError):
        layer.rope(q, f, pos0=1.5)


def test_sizes_past_32_bits_are_refused(fake_layer):
    """Sequences, tokens, channels and heads of 2^31 and more (of expanded tensors: no memory is needed), and a
    position past 2^53: refused, not taken by their remainder."""
    import preconditioned_delta_rule_token_b200 as pk
    layer, calls = fake_layer
    n = (1 << 32) + 5
    x = lambda *s: _fake(1, 1, 8).expand(*s)  # noqa: E731
    head = lambda *s: _fake(1, 1, 1, 8).expand(*s)  # noqa: E731
    f = _fake(4, dtype=torch.float64)
    for call in (lambda: layer.recurrence(x(1, n, 8), x(1, n, 8)), lambda: layer.recurrence(x(n, 1, 8), x(n, 1, 8)),
                 lambda: layer.recurrence_backward(x(1, n, 8), x(1, n, 8), x(1, n, 8)),
                 lambda: layer.recurrence_step(x(1, n, 8)[0], x(1, n, 8)[0], _fake(5, 8)),
                 lambda: layer.qk_norm(head(1, n, 1, 8), None), lambda: layer.qk_norm(head(n, 1, 1, 8), None),
                 lambda: layer.qk_norm(head(1, 2, 1, 8), head(1, 2, n, 8)), lambda: layer.rope(head(1, 2, n, 8), f),
                 lambda: layer.rope(head(1, 2, 1, 8), _fake(1, dtype=torch.float64).expand(n))):
        with pytest.raises(pk.OsdnError, match="below 2\\^31"):
            call()
    for pos0 in (1 << 64, (1 << 53) + 1, -(1 << 53) - 1):
        with pytest.raises(pk.OsdnError, match="pos0"):
            layer.rope(_fake(1, 2, 1, 8), f, pos0=pos0)
    assert not calls.reached


def test_no_key_heads_leave_a_zero_weight_gradient(fake_layer, monkeypatch):
    """k [B,T,0,width] with a weight: an empty dk, and dwk the sum over no rows."""
    layer, calls = fake_layer
    monkeypatch.setattr(calls, "like", lambda t: torch.full(t.shape, 7.0))
    q, k, w = _fake(1, 2, 3, 64), _fake(1, 2, 0, 64), _fake(64)
    g = layer.qk_norm_backward(q, k, q, k, wq=w, wk=w, workspace=_fake(1 << 12))
    assert g["dk"].shape == (1, 2, 0, 64) and bool((g["dwk"] == 0).all())


def test_a_step_reads_one_row_for_the_batch(fake_layer):
    """The strides that reach the library: 0 over the sequences, beside one that says that this is not the dense layout."""
    layer, calls = fake_layer
    x, one, state = _fake(3, 8), _fake(1, 8).expand(3, 8), _fake(3, 8)
    for a, b in ((x, one), (one, x), (one, one)):
        layer.recurrence_step(a, b, state)
        p = layer.B.osdn_recur_params.from_address(calls.reached[-1][1])
        for t, strides in ((a, p.stride_x), (b, p.stride_gate)):
            assert tuple(strides) == ((0, 8) if t is one else (0, 0))
        assert tuple(p.stride_h) == (0, 0)


def test_the_extension_module_belongs_to_this_torch(osdn_lib):
    """It is compiled against torch's C++ headers, so another torch has to get another file, and not load this one."""
    import os
    assert torch.__version__ in os.path.basename(osdn_lib.CALL_PATH)
    osdn_lib.build_call()
    assert os.path.exists(osdn_lib.CALL_PATH) and osdn_lib.call().layouts(None) == (-1).to_bytes(8, "little", signed=True)


# ------------------------------------------------------------------ GPU: the recurrence

@pytest.mark.gpu
@pytest.mark.parametrize("gdt", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("D", (16, 33))
def test_log_gates_below_the_normal_range(gdt, D):
    """With the norm scale 1 - a^2 = -2 gate: below the normal range it counts as 0, with the slope of s, so such
    a gate gives bit for bit what a gate of 0 gives; just inside the range the gradients are the formula's."""
    import preconditioned_delta_rule_token_b200 as pk
    g = torch.Generator().manual_seed(1)
    dt = gdt
    x, dh = torch.randn(2, 70, D, generator=g).to(dt), torch.randn(2, 70, D, generator=g).to(dt)
    h0, dfinal = torch.randn(2, D, generator=g), torch.randn(2, D, generator=g)
    base = -torch.rand(2, 70, D, generator=g) - 0.1
    pick = torch.randint(0, 12, (2, 70, D), generator=g)
    low = base.clone()
    for i, v in enumerate((-1e-39, -1e-40, -1e-45, float(torch.nn.functional.logsigmoid(torch.tensor(89.0))))):
        low[pick == i] = v
    low, zero = low.to(gdt), torch.where(pick < 4, 0.0, base).to(gdt)
    assert bool(((low != 0) & (low.float().abs() < 5e-39)).any())        # the type keeps them
    how = dict(gate_form="log", input_scale="norm")

    def run(gate):
        gate = gate.cuda()
        h, f, marks = pk.recurrence(x.cuda(), gate, h0=h0.cuda(), checkpoints=True, **how)
        r = pk.recurrence_backward(x.cuda(), gate, dh.cuda(), h0=h0.cuda(), dfinal_h=dfinal.cuda(), checkpoints=marks, **how)
        state = h0.cuda()
        return [h, f, r["dx"], r["dgate"], r["dh0"], pk.recurrence_step(x[:, 0].cuda(), gate[:, 0], state, **how), state]

    a, b = run(low), run(zero)
    assert all(bool(torch.isfinite(t).all()) for t in a)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    near = torch.where(pick < 4, -1e-38, base).to(gdt)                   # 1 - a^2 = 2e-38, a normal number
    got, want = run(near), ref.recurrence_grads(x, near, dh, h0, dfinal, None, "log", "norm")
    for t, k in zip(got[2:5], ("dx", "dgate", "dh0")):
        ref.close(t, *want[k], 24 * 70 + 96, k)


@pytest.mark.gpu
@pytest.mark.parametrize("types", ((torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)))
@pytest.mark.parametrize("B,T,D", ((7, 200, 24), (7, 200, 33), (7, 200, 34), (2, 2049, 72), (200, 70, 512)))
def test_saved_states_behind_a_length(types, B, T, D):
    """checkpoints[b, i] is the state before token 64 i, and behind the length the final state; the others are
    those of the same sequence without lengths."""
    import preconditioned_delta_rule_token_b200 as pk
    g = torch.Generator().manual_seed(9)
    dt, gdt = types
    x, gate = torch.randn(B, T, D, generator=g).to(dt).cuda(), torch.rand(B, T, D, generator=g).to(gdt).cuda()
    h0 = torch.randn(B, D, generator=g).cuda()
    lengths = torch.tensor(([0, 1, 64, 65, 128, T, T + 9] * B)[:B], dtype=torch.int32)
    for h in (None, torch.empty_like(x)):
        _, final, marks = pk.recurrence(x, gate, h0=h0, lengths=lengths.cuda(), h=h, checkpoints=True)
        whole = pk.recurrence(x, gate, h0=h0, checkpoints=True)[2]
        for b in range(B):
            first = (min(int(lengths[b]), T) + 63) // 64          # the first state behind the length
            assert torch.equal(marks[b, :first], whole[b, :first])
            assert torch.equal(marks[b, first:], final[b].expand_as(marks[b, first:]))


@pytest.mark.gpu
@pytest.mark.parametrize("types", ((torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32)))
@pytest.mark.parametrize("B,D", ((5, 64), (3, 33), (4, 1), (1, 8)))
def test_a_step_with_one_row_for_the_batch(types, B, D):
    """x or gate expanded over the sequences, as recurrence reads them: the values of the tensor in memory."""
    import preconditioned_delta_rule_token_b200 as pk
    g = torch.Generator().manual_seed(10)
    dt, gdt = types
    x, gate = torch.randn(B, D, generator=g).to(dt).cuda(), torch.randn(B, D, generator=g).to(gdt).cuda()
    h0 = torch.randn(B, D, generator=g).cuda()
    for a, b in ((x, gate[:1].expand(B, D)), (x[:1].expand(B, D), gate), (x[-1:].expand(B, D), gate[-1:].expand(B, D))):
        s, t = h0.clone(), h0.clone()
        got = pk.recurrence_step(a, b, s, gate_form="logit")
        assert torch.equal(got, pk.recurrence_step(a.contiguous(), b.contiguous(), t, gate_form="logit"))
        assert torch.equal(s, t)
    if B > 1:
        with pytest.raises(pk.OsdnError):        # a result for each sequence needs its own row
            pk.recurrence_step(x, gate, h0.clone(), out=torch.empty_like(x[:1]).expand(B, D))
        if D > 1:
            with pytest.raises(pk.OsdnError):
                pk.recurrence_step(x, gate[:1, :1].expand(B, D), h0.clone())


# ------------------------------------------------------------------ GPU: the norms

@pytest.mark.gpu
@pytest.mark.parametrize("dt", (torch.bfloat16, torch.float32))
@pytest.mark.parametrize("width", (40, 64, 128, 256))
@pytest.mark.parametrize("norm", ("l2", "rms"))
def test_a_nan_fills_its_row(dt, width, norm):
    """The norm divides by a sum over the row, so one NaN makes the whole row NaN, forward and backward, and
    no other row."""
    import preconditioned_delta_rule_token_b200 as pk
    g = torch.Generator().manual_seed(2)
    q, dq = (torch.randn(2, 9, 5, width, generator=g).to(dt).cuda() for _ in range(2))
    bad = torch.zeros(2, 9, 5, dtype=torch.bool)
    bad[0, 0, 0] = bad[0, 3, 4] = bad[1, 8, 2] = True
    bad = bad.cuda()
    x = q.clone()
    x[..., 7][bad] = float("nan")
    how = dict(freqs=ref.plain_freqs(16).cuda(), norm=norm)
    out, want = pk.qk_norm(x, x, **how), pk.qk_norm(q, q, **how)
    got, grad = pk.qk_norm_backward(x, x, dq, dq, **how), pk.qk_norm_backward(q, q, dq, dq, **how)
    for a, b in ((out[0], want[0]), (out[1], want[1]), (got["dq"], grad["dq"]), (got["dk"], grad["dk"])):
        assert bool(a[bad].isnan().all()) and torch.equal(a[~bad], b[~bad])


@pytest.mark.gpu
def test_an_infinity_keeps_to_its_row():
    """x / sqrt(infinity): NaN in the infinity's place (without rotation), zeros beside it."""
    import preconditioned_delta_rule_token_b200 as pk
    q = torch.randn(1, 4, 2, 64, generator=torch.Generator().manual_seed(3)).cuda()
    want = pk.qk_norm(q, None)[0]
    q[0, 2, 1, 9] = float("inf")
    out = pk.qk_norm(q, None)[0]
    row = torch.zeros(64, device="cuda")
    row[9] = float("nan")
    assert torch.equal(out[0, 2, 1].isnan(), row.isnan()) and bool((out[0, 2, 1].nan_to_num() == 0).all())
    want[0, 2, 1] = out[0, 2, 1] = 0
    assert torch.equal(out, want)


# ------------------------------------------------------------------ GPU: the calls together

@pytest.mark.gpu
@pytest.mark.parametrize("gated", (False, True))
def test_training_step_on_another_stream(gated):
    """forward() and backward() with qk on a side stream that is still busy, while the current stream allocates and
    writes: the results are those of the calls on the current stream. The forward's are bit for bit the same; the
    delta rule's backward sums in an order that may change, so its gradients are compared as its own tests do."""
    import preconditioned_delta_rule_token_b200 as pk
    B, T, H, W = 2, 256, 4, 128
    g = torch.Generator().manual_seed(5)
    new = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v, dout, beta = new(B, T, H, W), new(B, T, H, W), new(B, T, H, W), new(B, T, H, W), new(B, T, H).sigmoid()
    alpha = torch.sigmoid(3 + new(B, T, H)) if gated else None
    qk = pk.QkNorm(norm="rms", wq=torch.ones(W, device="cuda"), freqs=pk.rope_frequencies(W)[0], scale_k=W ** -0.5)

    def run(stream):
        out = pk.forward(q, k, v, beta, alpha=alpha, qk=qk, eta=0.1, stream=stream)
        grads = pk.backward(q, k, v, beta, dout, alpha=alpha, qk=qk, eta=0.1, stream=stream)
        return [*out, *(t for t in grads.values() if t is not None)]

    want = run(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)            # about 10 ms
        got = run(side)
        junk = [torch.full((B, T, H, W), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        junk += [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 20, 1 << 22, 1 << 24, 1 << 26)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[:3], got))
        for a, b in zip(want[3:], got[3:]):
            assert float((a.double() - b.double()).abs().max()) <= BF16_TOL * float(a.double().abs().max())
        del junk


@pytest.mark.gpu
def test_workspaces_of_the_caller():
    """A given workspace gives what an own one gives; one that is too small is refused by the library."""
    import preconditioned_delta_rule_token_b200 as pk
    g = torch.Generator().manual_seed(6)
    x, gate, dh = (torch.randn(2, 150, 40, generator=g).cuda() for _ in range(3))
    q, w = torch.randn(2, 50, 4, 64, generator=g).cuda(), torch.ones(64, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    a = pk.recurrence_backward(x, gate, dh, gate_form="logit")
    b = pk.recurrence_backward(x, gate, dh, gate_form="logit", workspace=ws)
    c = pk.qk_norm_backward(q, q, q, q, wq=w, wk=w)
    d = pk.qk_norm_backward(q, q, q, q, wq=w, wk=w, workspace=ws)
    assert all(torch.equal(a[n], b[n]) for n in a) and all(torch.equal(c[n], d[n]) for n in c)
    for call in (lambda: pk.recurrence_backward(x, gate, dh, gate_form="logit", workspace=ws[:64]),
                 lambda: pk.qk_norm_backward(q, q, q, q, wq=w, workspace=ws[:64])):
        with pytest.raises(pk.OsdnError, match="too small"):
            call()


@pytest.mark.gpu
def test_a_scale_that_changes_in_place():
    import preconditioned_delta_rule_token_b200 as pk
    q = torch.randn(1, 3, 2, 64, generator=torch.Generator().manual_seed(7)).cuda()
    s = torch.tensor(1.0)
    a = pk.qk_norm(q, None, scale_q=s)[0]
    s.fill_(2.0)
    assert torch.equal(pk.qk_norm(q, None, scale_q=s)[0], 2 * a)


@pytest.mark.gpu
def test_no_key_heads():
    import preconditioned_delta_rule_token_b200 as pk
    q, w = torch.randn(1, 3, 2, 64, generator=torch.Generator().manual_seed(8)).cuda(), torch.ones(64, device="cuda")
    k = q[:, :, :0].contiguous()
    out, got = pk.qk_norm(q, k, wq=w, wk=w), pk.qk_norm_backward(q, k, q, k, wq=w, wk=w)
    want = pk.qk_norm_backward(q, None, q, None, wq=w)
    assert torch.equal(out[0], pk.qk_norm(q, None, wq=w)[0]) and out[1].shape == got["dk"].shape == (1, 3, 0, 64)
    assert torch.equal(got["dq"], want["dq"]) and torch.equal(got["dwq"], want["dwq"]) and bool((got["dwk"] == 0).all())


@pytest.mark.gpu
def test_a_step_larger_than_its_grid():
    """More channels than threads at a time (eight blocks of 256 an SM, four channels or one a thread)."""
    import preconditioned_delta_rule_token_b200 as pk
    g = torch.Generator(device="cuda").manual_seed(11)
    for B, D in ((700, 4096), (700, 1001)):
        x, gate, state = (torch.randn(B, D, generator=g, device="cuda") for _ in range(3))
        rows = state.clone()
        out = pk.recurrence_step(x, gate, rows, gate_form="logit", input_scale="complement")
        for i in (0, 1, B // 2, B - 1):              # each sequence alone gives the same bits
            one = state[i:i + 1].clone()
            want = pk.recurrence_step(x[i:i + 1], gate[i:i + 1], one, gate_form="logit", input_scale="complement")
            assert torch.equal(out[i:i + 1], want) and torch.equal(rows[i:i + 1], one)
        a = torch.sigmoid(gate.double())
        h = a * state.double() + (1 - a) * x.double()
        # 12 + 48 roundings of the terms, as for one token in test_recurrence.py
        assert bool(((rows.double() - h).abs() <= 60 * 2.0 ** -24 * (a * state.double().abs() + x.double().abs())).all())


@pytest.mark.gpu
def test_captured_training_step_and_decode_token():
    """forward(), backward() and step() with qk captured into a graph and replayed with new inputs."""
    import preconditioned_delta_rule_token_b200 as pk
    B, T, H, W = 2, 192, 3, 128
    g = torch.Generator().manual_seed(12)
    new = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v, dout, beta = new(B, T, H, W), new(B, T, H, W), new(B, T, H, W), new(B, T, H, W), new(B, T, H).sigmoid()
    q2, k2 = new(B, T, H, W), new(B, T, H, W)
    qk = pk.QkNorm(norm="rms", wq=torch.ones(W, device="cuda"), wk=torch.ones(W, device="cuda"),
                   freqs=pk.rope_frequencies(W)[0], scale_k=W ** -0.5)
    at = torch.full((B,), T, device="cuda")

    def run():
        out, S, d = pk.forward(q, k, v, beta, qk=qk, eta=0.1)
        grads = pk.backward(q, k, v, beta, dout, qk=qk, eta=0.1)
        token = pk.step(*(t[:, 0].contiguous() for t in (q, k, v, beta)), S, d, eta=0.1, qk=qk, positions=at)
        return [out, S, d, token], [t for t in grads.values() if t is not None]

    first = [t.clone() for t in (q, k)]
    want = run()
    q.copy_(q2), k.copy_(k2)
    want2 = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for (a, b), exp in (((q2, k2), want2), (first, want)):
        q.copy_(a), k.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(exp[0], got[0]))
        for x, y in zip(exp[1], got[1]):
            assert float((x.double() - y.double()).abs().max()) <= BF16_TOL * float(x.double().abs().max())


@pytest.mark.gpu
def test_two_training_steps_at_once():
    """forward() and backward() with qk in flight on two streams at a time give what they give alone."""
    import preconditioned_delta_rule_token_b200 as pk
    B, T, H, W = 2, 192, 3, 128
    qk = pk.QkNorm(wq=torch.ones(W, device="cuda"), freqs=pk.rope_frequencies(W)[0])
    cases = []
    for seed in (13, 14):
        g = torch.Generator().manual_seed(seed)
        cases.append([torch.randn(B, T, H, W, generator=g).bfloat16().cuda() for _ in range(4)] +
                     [torch.rand(B, T, H, generator=g).bfloat16().cuda()])

    def run(c, stream):
        q, k, v, dout, beta = c
        out = pk.forward(q, k, v, beta, qk=qk, eta=0.1, stream=stream)
        grads = pk.backward(q, k, v, beta, dout, qk=qk, eta=0.1, stream=stream)
        return list(out), [t for t in grads.values() if t is not None]

    want = [run(c, None) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(c, s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
        for x, y in zip(a[1], b[1]):
            assert float((x.double() - y.double()).abs().max()) <= BF16_TOL * float(x.double().abs().max())
