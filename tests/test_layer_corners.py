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
