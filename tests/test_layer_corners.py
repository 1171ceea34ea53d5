"""Corners of the layer's operators: gates below the normal range, rows with NaN, temporaries of a call on another
stream, host tensors at the raw entry points, and other calls that the documentation allows or has to refuse.

Tolerances are those of test_recurrence.py and test_qk_norm.py, counted in roundings there."""
import pytest
import torch

from tests import _layer_ref as ref


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
