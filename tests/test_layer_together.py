"""The operators as a layer uses them: fused projection -> norms of q and k with the rotation ->
(gated) delta rule -> gated linear recurrence over its outputs, as prefill, as training step and token
by token.

What the delta rule's own tests allow (2e-2 of the largest value of a sequence and head in bf16, 1e-4 in
fp32) holds for the chain too: the norms' outputs enter the oracle as the kernel rounded them, so the chain
adds no error of its own before the delta rule; the norms' backward multiplies the delta rule's
gradients by a map of norm at most 2 / |x|, and is compared on the same scale.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from tests import _layer_ref as ref
from tests._util import BF16_TOL, FP32_TOL, slice_rel_err

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _inputs(seed, B, T, H, dk, dv, dt, gated):
    g = torch.Generator().manual_seed(seed)
    fused = torch.randn(B, T, H, 2 * dk + dv, generator=g).to(dt).cuda()
    beta = torch.sigmoid(torch.randn(B, T, H, generator=g)).to(dt).cuda()
    alpha = torch.sigmoid(3 + torch.randn(B, T, H, generator=g)).to(dt).cuda() if gated else None
    return fused[..., :dk], fused[..., dk:2 * dk], fused[..., 2 * dk:], beta, alpha


def _f(t):
    return None if t is None else np.ascontiguousarray(ref.f64(t).numpy())


def _options(pk, dk, weights):
    freqs, amp = pk.rope_frequencies(dk // 2, scaling="linear", factor=2.0)
    w = (lambda s: 1 + 0.1 * torch.randn(dk, generator=torch.Generator().manual_seed(s)).cuda()) if weights else lambda s: None
    # with RMS weights the keys keep length 1 through scale_k
    return pk.QkNorm(norm="rms" if weights else "l2", wq=w(1), wk=w(2), freqs=freqs, amplitude=amp,
                     scale_k=dk ** -0.5 if weights else 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,gated,weights", ((torch.bfloat16, True, False), (torch.bfloat16, False, True),
                                              (torch.float32, False, True)))
def test_training_step(dt, gated, weights):
    """forward() and backward() with qk equal the operators called one by one bit for bit, and the gradients of
    the raw q and k are the oracle's for the chain."""
    import preconditioned_delta_rule_token_b200 as pk
    B, T, H, dk, dv = 2, 150, 3, 128, 128
    q, k, v, beta, alpha = _inputs(1, B, T, H, dk, dv, dt, gated)
    v = v.contiguous()
    qk = _options(pk, dk, weights)
    pos = ref.positions_of(B, T, 77).cuda()
    out, S, d = pk.forward(q, k, v, beta, alpha=alpha, qk=qk, positions=pos, eta=0.1)
    qn, kn = qk.apply(q, k, pos)
    one = pk.forward(qn, kn, v, beta, alpha=alpha, eta=0.1)
    assert all(torch.equal(a, b) for a, b in zip((out, S, d), one))
    tol = BF16_TOL if dt == torch.bfloat16 else FP32_TOL
    want = oracle.fwd(_f(qn), _f(kn), _f(v), _f(beta), None, None, None, eta=0.1, alpha=_f(alpha))
    assert slice_rel_err(ref.f64(out).numpy(), want[0], (0, 2)) < tol

    # the recurrence over the layer's outputs, its gradient into the delta rule's backward
    x = out.view(B, T, H * dv)
    gate = torch.randn(B, T, H * dv, generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    dh = torch.randn(B, T, H * dv, generator=torch.Generator().manual_seed(4)).to(dt).cuda()
    how = dict(gate_form="logit", input_scale="complement")
    h, _, marks = pk.recurrence(x, gate, checkpoints=True, **how)
    want_h, _, mag, _ = ref.recurrence(x, gate, None, None, "logit", "complement")
    ref.close(h, want_h, mag, 12 * T + 48, "h")
    dx = pk.recurrence_backward(x, gate, dh, checkpoints=marks, **how)["dx"]
    g = pk.backward(q, k, v, beta, dx.view(B, T, H, dv), alpha=alpha, qk=qk, positions=pos, eta=0.1)
    w = oracle.bwd(_f(qn), _f(kn), _f(v), _f(beta), _f(dx.view(B, T, H, dv)), None, None, None, None, None, eta=0.1,
                   alpha=_f(alpha))
    for name, raw, wt, scale in (("dq", q, qk.wq, qk.scale_q), ("dk", k, qk.wk, qk.scale_k)):
        (dwant, _), dw = ref.head_norm_grads(raw, wt, torch.from_numpy(w[name]), qk.norm, qk.eps, scale, qk.freqs.cpu(),
                                             pos.cpu(), qk.layout, qk.amplitude)
        assert slice_rel_err(ref.f64(g[name]).numpy(), dwant.numpy(), (0, 2)) < 2 * tol, name
        if weights:
            assert slice_rel_err(ref.f64(g["dw" + name[1]]).numpy()[None], dw[0].numpy()[None], (0,)) < 2 * tol
        else:
            assert g["dw" + name[1]] is None
    assert slice_rel_err(ref.f64(g["dv"]).numpy(), w["dv"], (0, 2)) < tol
    assert pk.osdn_sync_status() == 0


@pytest.mark.gpu
def test_prefill_then_tokens():
    """Prefill and decode give what one prefill over all tokens gives: the rotation goes on at each sequence's
    own position, the delta rule and the recurrence from their states."""
    import preconditioned_delta_rule_token_b200 as pk
    B, T, n, H, dk, dv = 3, 70, 4, 2, 128, 128
    q, k, v, beta, alpha = _inputs(5, B, T + n, H, dk, dv, torch.bfloat16, True)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qk = _options(pk, dk, True)
    start = torch.tensor([0, 1000, 200000]).cuda()
    pos = start[:, None] + torch.arange(T + n).cuda()[None]
    gate = torch.randn(B, T + n, H * dv, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    how = dict(gate_form="logit", input_scale="norm")
    full, _, _ = pk.forward(q, k, v, beta, alpha=alpha, qk=qk, positions=pos, eta=0.1)
    full_h, full_state = pk.recurrence(full.view(B, T + n, H * dv), gate, **how)
    cut = lambda t: t[:, :T].contiguous()  # noqa: E731
    out, S, d = pk.forward(cut(q), cut(k), cut(v), cut(beta), alpha=cut(alpha), qk=qk, positions=cut(pos), eta=0.1)
    h, state = pk.recurrence(out.view(B, T, H * dv), cut(gate), **how)
    assert torch.equal(h, full_h[:, :T])
    for t in range(T, T + n):
        tok = lambda x: x[:, t].contiguous()  # noqa: E731
        o = pk.step(tok(q), tok(k), tok(v), tok(beta), S, d, eta=0.1, alpha=tok(alpha), qk=qk, positions=tok(pos))
        hs = pk.recurrence_step(o.view(B, H * dv), gate[:, t], state, **how)
        assert slice_rel_err(ref.f64(o).numpy(), ref.f64(full[:, t]).numpy(), (0, 1)) < BF16_TOL
        assert slice_rel_err(ref.f64(hs).numpy(), ref.f64(full_h[:, t]).numpy(), (0,)) < BF16_TOL
    assert slice_rel_err(ref.f64(state).numpy(), ref.f64(full_state).numpy(), (0,)) < BF16_TOL


@pytest.mark.gpu
def test_two_streams_at_once():
    """Two training steps in flight on two streams, each with its own temporaries, give what they give alone."""
    import preconditioned_delta_rule_token_b200 as pk
    qk = _options(pk, 128, True)
    cases = []
    for s in (7, 8):
        q, k, v, beta, _ = _inputs(s, 2, 256, 4, 128, 128, torch.bfloat16, False)
        cases.append((q, k, torch.randn_like(q), *(t.reshape(2, 256, 512) for t in (q, k))))
    run = lambda c, st: [*qk.apply(c[0], c[1], None, st),  # noqa: E731
                         *(t for t in qk.gradients(c[0], c[1], c[2], c[2], None, st).values()),
                         *pk.recurrence(c[3], c[4], gate_form="logit", stream=st)]
    want = [run(c, None) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got = [run(c, st) for c, st in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_positions_need_the_norm():
    import preconditioned_delta_rule_token_b200 as pk
    x, b = torch.zeros(1, 4, 1, 64), torch.zeros(1, 4, 1)
    for call in (lambda: pk.forward(x, x, x, b, positions=b), lambda: pk.backward(x, x, x, b, x, positions=b),
                 lambda: pk.step(x[:, 0], x[:, 0], x[:, 0], b[:, 0], x, x, positions=b)):
        with pytest.raises(pk.OsdnError, match="positions"):
            call()


_FIRST_IN_A_CAPTURE = """
import torch
import preconditioned_delta_rule_token_b200 as pk
x = torch.randn(2, 300, 64, device="cuda").bfloat16()
q = torch.randn(2, 300, 2, 64, device="cuda").bfloat16()
w, f = torch.ones(64, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda")
def run():
    h, s, m = pk.recurrence(x, x, gate_form="logit", checkpoints=True)
    g = pk.recurrence_backward(x, x, x, checkpoints=m, gate_form="logit")
    o = pk.recurrence_step(x[:, 0], x[:, 0], s.clone(), gate_form="logit")
    n = pk.qk_norm(q, q, freqs=f, wq=w)
    d = pk.qk_norm_backward(q, q, q, q, freqs=f, wq=w)
    return [h, s, g["dx"], g["dgate"], o, *n, d["dq"], d["dwq"], pk.rope(q, f)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
print("same")
"""


@pytest.mark.gpu
def test_first_calls_of_a_process_inside_a_capture():
    """Nothing has to run before a capture: the kernels' limits and the room on the device are asked for on the host."""
    r = subprocess.run([sys.executable, "-c", _FIRST_IN_A_CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_raw_calls_equal_the_wrappers():
    """The C entry points through the ctypes binding, with everything preallocated."""
    import ctypes

    import preconditioned_delta_rule_token_b200 as pk
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s, dt=torch.bfloat16: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, gate, dh, h0 = new(2, 200, 64), new(2, 200, 64), new(2, 200, 64), new(2, 64, dt=torch.float32)
    p = pk.osdn_recur_params()
    p.struct_size, p.B, p.T, p.D, p.gate_form = ctypes.sizeof(p), 2, 200, 64, 2
    h, f, m = torch.empty_like(x), torch.empty_like(h0), torch.empty(2, 4, 64, device="cuda")
    pk.osdn_recur_fwd(p, x, gate, h0, None, h, f, m)
    want = pk.recurrence(x, gate, h0=h0, gate_form="logit", checkpoints=True)
    assert all(torch.equal(a, b) for a, b in zip((h, f, m), want))
    dx, dg, d0 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(h0)
    ws = torch.empty(pk.osdn_recur_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    pk.osdn_recur_bwd(p, x, gate, h0, None, dh, None, None, dx, dg, d0, ws)
    grads = pk.recurrence_backward(x, gate, dh, h0=h0, checkpoints=m, gate_form="logit")
    assert all(torch.equal(a, grads[k]) for a, k in ((dx, "dx"), (dg, "dgate"), (d0, "dh0")))
    s1, s2, o = f.clone(), f.clone(), torch.empty_like(x[:, 0].contiguous())
    p.stride_x[0] = p.stride_gate[0] = 200 * 64
    pk.osdn_recur_step(p, x, gate, s1, o)
    assert torch.equal(o, pk.recurrence_step(x[:, 0], gate[:, 0], s2, gate_form="logit")) and torch.equal(s1, s2)

    q, k, w = new(2, 30, 4, 64), new(2, 30, 2, 64), new(64, dt=torch.float32)
    fr = torch.tensor(pk.osdn_rope_freqs(32, 10000.0, 0, 1.0, 0, 1.0, 4.0)[0], dtype=torch.float64, device="cuda")
    p = pk.osdn_qk_params()
    p.struct_size, p.B, p.T, p.Hq, p.Hk, p.width, p.norm, p.rot_dim = ctypes.sizeof(p), 2, 30, 4, 2, 64, 2, 32
    p.eps, p.amplitude, p.scale_q, p.scale_k, p.pos0 = 1e-6, 1.0, 1.0, 1.0, 5
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pk.osdn_qk_fwd(p, q, k, w, w, None, fr, None, qo, ko)
    how = dict(freqs=fr, norm="rms", wq=w, wk=w, pos0=5)
    assert all(torch.equal(a, b) for a, b in zip((qo, ko), pk.qk_norm(q, k, **how)))
    dq, dk, dwq, dwk = torch.empty_like(q), torch.empty_like(k), torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(pk.osdn_qk_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    pk.osdn_qk_bwd(p, q, k, w, w, None, fr, None, qo, ko, dq, dk, dwq, dwk, ws)
    grads = pk.qk_norm_backward(q, k, qo, ko, **how)
    assert all(torch.equal(a, grads[n]) for a, n in ((dq, "dq"), (dk, "dk"), (dwq, "dwq"), (dwk, "dwk")))
    p.norm = 0
    pk.osdn_rope(p, q, None, fr, None, qo, inverse=True)
    assert torch.equal(qo, pk.rope(q, fr, pos0=5, inverse=True))
