"""Norms of queries and keys for each head with the position rotation, their backward, and the
rotation alone.

Tolerances, fixed before the first run, in fp32 roundings of the sum of absolute terms (plus half a
step of the output's type). The sum of squares of up to 256 features in 8 by lane and 5 between lanes
takes 14 and counts half through the root; root and quotient 4; scale, weight and their products 4; a
cosine carries 2^-25 of an angle of up to pi from its fraction and 2 units of its own, together 8, and the
turn 3: 32 in all. The gradient has two such chains and a dot product over the row: 96. The weights'
gradient adds one term a row on top: rows + 96."""
import ctypes
import math

import pytest
import torch

from tests import _layer_ref as ref

BF, FP = torch.bfloat16, torch.float32


def rows(seed, B, T, H, W, dt):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(B, T, H, W, generator=g).to(dt), torch.randn(B, T, H, W, generator=g).to(dt)


# ------------------------------------------------------------------ CPU: the formulas, the frequencies, the refusals

@pytest.mark.parametrize("norm", ("none", "l2", "rms"))
@pytest.mark.parametrize("layout", ("half", "interleaved"))
def test_the_gradient_formulas_agree_with_differences(norm, layout):
    x, dout = (t.double() for t in rows(1, 1, 3, 2, 16, FP))
    w = None if norm == "none" else 1 + 0.1 * torch.randn(16, dtype=torch.float64, generator=torch.Generator().manual_seed(2))
    pos, fr = ref.positions_of(1, 3, 5), ref.plain_freqs(8)
    a = (norm, 1e-3, 0.7, fr, pos, layout, 1.2)

    def loss(x, w):
        return float((ref.head_norm(x, w, *a)[0] * dout).sum())

    (dx, _), dw = ref.head_norm_grads(x, w, dout, *a)
    for i in range(x.numel()):
        e = torch.zeros(x.numel(), dtype=torch.float64)
        e[i] = 1e-6
        e = e.view_as(x)
        assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-6 - float(dx.flatten()[i])) < 1e-6
    for i in range(16 if w is not None else 0):
        e = torch.zeros(16, dtype=torch.float64)
        e[i] = 1e-6
        assert abs((loss(x, w + e) - loss(x, w - e)) / 2e-6 - float(dw[0][i])) < 1e-6


def test_scaled_frequencies():
    """Each scaling against its definition written out: ends, ramp and amplitude."""
    import preconditioned_delta_rule_token_b200 as pk
    kw = dict(device="cpu")
    for rot in (2, 32, 64, 128):
        f, a = pk.rope_frequencies(rot, **kw)
        assert a == 1.0 and torch.allclose(f, ref.plain_freqs(rot), rtol=1e-14)
        assert torch.allclose(pk.rope_frequencies(rot, scaling="linear", factor=4, **kw)[0], f / 4, rtol=1e-14)
    plain = ref.plain_freqs(64)
    ntk, _ = pk.rope_frequencies(64, scaling="ntk", factor=8, **kw)
    assert ntk[0] == 1.0 and abs(float(plain[-1] / ntk[-1]) - 8) < 1e-12
    assert torch.allclose(ntk, ref.plain_freqs(64, 10000.0 * 8 ** (64 / 62)), rtol=1e-13)
    turns = 4096 * plain / (2 * math.pi)
    yarn, a = pk.rope_frequencies(64, scaling="yarn", factor=16, original_length=4096, **kw)
    assert abs(a - (0.1 * math.log(16) + 1)) < 1e-15
    at = [64 * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(10000)) for n in (32, 1)]
    low, high = math.floor(at[0]), math.ceil(at[1])
    for i in range(32):
        m = min(max((i - low) / (high - low), 0), 1)
        assert abs(float(yarn[i] / plain[i]) - (m / 16 + 1 - m)) < 1e-12
    assert bool((yarn[turns > 40] == plain[turns > 40]).all())
    wave, a = pk.rope_frequencies(64, scaling="wavelength", factor=8, original_length=4096, **kw)
    assert a == 1.0
    for i in range(32):
        m = min(max((float(turns[i]) - 1) / 3, 0), 1)
        assert abs(float(wave[i] / plain[i]) - ((1 - m) / 8 + m)) < 1e-12
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=512), dict(base=1.0), dict(base=float("nan")),
                dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=2.0), dict(scaling="other"),
                dict(scaling="ntk", factor=2.0, rot_dim=2),
                dict(scaling="wavelength", factor=2.0, original_length=100, low_turns=4.0)):
        with pytest.raises(pk.OsdnError):
            pk.rope_frequencies(**{**dict(rot_dim=64, device="cpu"), **bad})


def _params(lib_, **kw):
    p = lib_.osdn_qk_params()
    p.struct_size = ctypes.sizeof(p)
    a = dict(B=2, T=10, Hq=4, Hk=2, width=128, dtype=0, norm=2, layout=0, rot_dim=64, eps=1e-6, amplitude=1.0,
             scale_q=1.0, scale_k=1.0)
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
    inv, uns, nan = B.OSDN_ERR_INVALID_ARG, B.OSDN_ERR_UNSUPPORTED, float("nan")
    assert ctypes.sizeof(B.osdn_qk_params) == 168
    assert L.osdn_qk_bwd_workspace_size(_params(B), ctypes.byref(n)) == 0 and n.value >= 2 * 128 * 4
    for kw, code in ((dict(B=0), inv), (dict(T=-1), inv), (dict(Hq=0), inv), (dict(Hk=-1), inv), (dict(width=0), inv),
                     (dict(width=100), uns), (dict(width=264, rot_dim=0), uns), (dict(dtype=5), inv), (dict(norm=3), inv),
                     (dict(layout=2), inv), (dict(rot_dim=63), inv), (dict(rot_dim=130), inv), (dict(rot_dim=20), uns),
                     (dict(eps=-1.0), inv), (dict(eps=nan), inv), (dict(amplitude=nan), inv),
                     (dict(scale_q=float("inf")), inv), (dict(stride_q=(4, 0, 0)), inv),
                     (dict(stride_out_k=(-8, 8, 8)), inv), (dict(B=1 << 20, T=1 << 20), inv), (dict(reserved=1), inv)):
        assert L.osdn_qk_bwd_workspace_size(_params(B, **kw), ctypes.byref(n)) == code, kw
        assert B.get_last_error()


def test_pointers_are_checked_on_the_host(osdn_lib):
    B, L = osdn_lib, osdn_lib.lib()
    inv = B.OSDN_ERR_INVALID_ARG
    f = [(1 << 20) + (i << 16) for i in range(12)]    # never dereferenced: the checks fail first

    def fwd(p=None, **kw):
        names = ("q", "k", "wq", "wk", "positions", "freqs", "lengths", "q_out", "k_out", "stream")
        d = dict(q=f[0], k=f[1], freqs=f[2], q_out=f[3], k_out=f[4])
        d.update(kw)
        return L.osdn_qk_fwd(p or _params(B), *[d.get(n) for n in names])

    for kw in (dict(q=None), dict(k=None), dict(freqs=None), dict(q_out=None), dict(k_out=None), dict(q=f[0] + 8),
               dict(wq=f[5] + 4), dict(positions=f[5] + 4), dict(q_out=f[1]), dict(k_out=f[0]), dict(k_out=f[3]),
               dict(p=_params(B, norm=0), wq=f[5]), dict(p=_params(B, stride_out_q=(0, 512, 128))),
               dict(p=_params(B, stride_q=(10240, 1024, 128)), q_out=f[0])):
        assert fwd(**kw) == inv, kw

    def bwd(p=None, **kw):
        names = ("q", "k", "wq", "wk", "positions", "freqs", "lengths", "dq_out", "dk_out", "dq", "dk", "dwq", "dwk",
                 "ws", "bytes", "stream")
        d = dict(q=f[0], k=f[1], freqs=f[2], dq_out=f[3], dk_out=f[4], dq=f[5], dk=f[6], bytes=0)
        d.update(kw)
        return L.osdn_qk_bwd(p or _params(B), *[d.get(n) for n in names])

    for kw in (dict(q=None), dict(dq=None), dict(dk_out=None), dict(dq=f[0]), dict(dk=f[4]), dict(dk=f[5]),
               dict(dwq=f[7]), dict(dwq=f[7], ws=f[8], bytes=64), dict(p=_params(B, norm=0), dwk=f[7])):
        assert bwd(**kw) == inv, kw
    assert L.osdn_rope(_params(B), f[0], None, f[2], None, f[3], 0, None) == inv            # a norm is set
    assert L.osdn_rope(_params(B, norm=0, rot_dim=0), f[0], None, f[2], None, f[3], 0, None) == inv
    assert L.osdn_rope(_params(B, norm=0), f[0], None, None, None, f[3], 0, None) == inv


def test_the_wrappers_refuse_what_they_cannot_take():
    import preconditioned_delta_rule_token_b200 as pk
    x = torch.zeros(1, 2, 3, 64)
    for call in (lambda: pk.qk_norm(x, x), lambda: pk.qk_norm(x[0], None), lambda: pk.rope(x, None),
                 lambda: pk.rope(x, torch.ones(32, dtype=torch.float64))):
        with pytest.raises(pk.OsdnError):
            call()


# ------------------------------------------------------------------ GPU

def _check_all(B, T, Hq, Hk, W, dt, norm, layout, rot, seed=1, start=0, amplitude=1.0, weights=True, eps=1e-6, lengths=None):
    import preconditioned_delta_rule_token_b200 as pk
    g = torch.Generator().manual_seed(100 + seed)
    (q, dq), (k, dk) = rows(seed, B, T, Hq, W, dt), rows(seed + 50, B, T, max(Hk, 1), W, dt)
    wq, wk = (1 + 0.1 * torch.randn(W, generator=g) if weights and norm != "none" else None for _ in range(2))
    fr = ref.plain_freqs(rot) if rot else None
    pos = ref.positions_of(B, T, start)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    how = dict(freqs=dev(fr), positions=pos.cuda(), norm=norm, eps=eps, wq=dev(wq), wk=dev(wk), layout=layout,
               amplitude=amplitude, scale_q=0.25)
    if not Hk:
        k = dk = how["wk"] = None
    qo, ko = pk.qk_norm(dev(q), dev(k), **how)
    got = pk.qk_norm_backward(dev(q), dev(k), dev(dq), dev(dk), **how)
    for x, w, do, out, s, n in ((q, wq, dq, qo, 0.25, "q"), (k, wk, dk, ko, 1.0, "k")):
        if x is None:
            assert out is None and got["dk"] is None and got["dwk"] is None
            continue
        a = (norm, eps, s, fr, pos, layout, amplitude)
        ref.close(out, *ref.head_norm(x, w, *a), 32, n)
        dx, dw = ref.head_norm_grads(x, w, do, *a)
        ref.close(got["d" + n], *dx, 96, "d" + n)
        if w is not None:
            ref.close(got["dw" + n], *dw, B * T * x.shape[2] + 96, "dw" + n)
        else:
            assert got["dw" + n] is None
    assert pk.osdn_sync_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("W", (8, 16, 40, 64, 96, 128, 200, 256))
@pytest.mark.parametrize("layout", ("half", "interleaved"))
@pytest.mark.parametrize("dt", (BF, FP))
def test_widths(W, layout, dt):
    rot = W
    _check_all(2, 5, 3, 2, W, dt, "rms", layout, rot, seed=W)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", ("none", "l2", "rms"))
@pytest.mark.parametrize("layout,rot", (("half", 8), ("half", 24), ("half", 64), ("interleaved", 6), ("interleaved", 62), ("half", 0)))
@pytest.mark.parametrize("weights", (False, True))
def test_norms_and_parts_of_the_head(norm, layout, rot, weights):
    _check_all(1, 9, 4, 1, 64, FP, norm, layout, rot, seed=3, start=70000, amplitude=1.2, weights=weights)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hq,Hk", ((1, 1, 1, 0), (1, 1, 16, 16), (70, 1, 5, 5), (3, 33, 32, 8), (2, 2100, 2, 1)))
@pytest.mark.parametrize("dt", (BF, FP))
def test_batches_and_heads(B, T, Hq, Hk, dt):
    _check_all(B, T, Hq, Hk, 128, dt, "l2", "half", 128, seed=4)


@pytest.mark.gpu
def test_far_positions_keep_their_angle():
    """Positions near 2^40 and negative ones: the angle is taken in 64 bits."""
    import preconditioned_delta_rule_token_b200 as pk
    x, _ = rows(5, 2, 6, 2, 64, FP)
    fr = ref.plain_freqs(64)
    pos = torch.tensor([[0, 1, -1, 1 << 20, (1 << 40) + 7, -(1 << 31)], [3, 1 << 24, 65535, -7, 12345678901, 2]])
    got = pk.rope(x.cuda(), fr.cuda(), positions=pos.cuda())
    want, mag = ref.turn(x.double(), pos, fr, "half", 1.0)
    # both sides form position * freq in 64 bits: 2^40 2^-53 of a radian apart at most, 2^-13
    far = (pos.abs() > (1 << 30))[..., None, None]
    ref.close(torch.where(far.cuda(), 0.0, got), torch.where(far, 0.0, want), mag, 32, "near")
    ref.close(got, want, mag, 32 + 2 ** 12, "far")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ("half", "interleaved"))
@pytest.mark.parametrize("dt", (BF, FP))
def test_the_rotation_alone_and_its_transpose(layout, dt):
    import preconditioned_delta_rule_token_b200 as pk
    x, do = rows(6, 2, 19, 3, 128, dt)
    fr, amp = pk.rope_frequencies(96, scaling="yarn", factor=4, original_length=2048)
    pos = ref.positions_of(2, 19, 1000)
    want, mag = ref.turn(x.double(), pos, fr.cpu(), layout, amp)
    got = pk.rope(x.cuda(), fr, positions=pos.cuda(), layout=layout, amplitude=amp)
    ref.close(got, want, mag, 32, "rope")
    assert torch.equal(got, pk.rope(x.cuda(), fr, pos0=1000, layout=layout, amplitude=amp))   # the same positions
    want, mag = ref.turn(do.double(), pos, fr.cpu(), layout, amp, -1.0)
    ref.close(pk.rope(do.cuda(), fr, positions=pos.cuda(), layout=layout, amplitude=amp, inverse=True), want, mag, 32,
              "transpose")
    y = x.cuda()
    assert pk.rope(y, fr, positions=pos.cuda(), layout=layout, amplitude=amp, out=y) is y and torch.equal(y, got)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", (BF, FP))
def test_in_place_and_fused_projections(dt):
    """q and k as column slices of one projection, written over themselves or into slices of another
    buffer: the same values as dense tensors, and v untouched."""
    import preconditioned_delta_rule_token_b200 as pk
    B, T, H, W = 2, 37, 3, 64
    q, dq = rows(7, B, T, H, W, dt)
    k, dk = rows(8, B, T, H, W, dt)
    how = dict(freqs=ref.plain_freqs(W).cuda(), norm="l2", pos0=3)
    want = pk.qk_norm(q.cuda(), k.cuda(), **how)
    fused = torch.full((B, T, H, 3 * W), 5.0, dtype=dt, device="cuda")
    qs, ks = fused[..., :W], fused[..., W:2 * W]
    qs.copy_(q), ks.copy_(k)
    other = torch.full((B, T, 3 * H, W), 9.0, dtype=dt, device="cuda")
    pk.qk_norm(qs, ks, q_out=other[:, :, :H], k_out=other[:, :, 2 * H:], **how)
    assert torch.equal(other[:, :, :H], want[0]) and torch.equal(other[:, :, 2 * H:], want[1])
    assert bool((other[:, :, H:2 * H] == 9.0).all())
    dfused = torch.zeros_like(fused)
    dfused[..., :W], dfused[..., W:2 * W] = dq.cuda(), dk.cuda()
    a = pk.qk_norm_backward(qs, ks, dfused[..., :W], dfused[..., W:2 * W], **how)
    b = pk.qk_norm_backward(q.cuda(), k.cuda(), dq.cuda(), dk.cuda(), **how)
    assert torch.equal(a["dq"], b["dq"]) and torch.equal(a["dk"], b["dk"])
    pk.qk_norm(qs, ks, q_out=qs, k_out=ks, **how)
    assert torch.equal(qs, want[0]) and torch.equal(ks, want[1]) and bool((fused[..., 2 * W:] == 5.0).all())


@pytest.mark.gpu
def test_one_query_for_every_head():
    """Heads expanded with stride 0 are read as they are; their gradient comes out for each head."""
    import preconditioned_delta_rule_token_b200 as pk
    q, dq = rows(9, 2, 11, 1, 64, FP)
    do = torch.randn(2, 11, 4, 64, generator=torch.Generator().manual_seed(1)).cuda()
    e = q.cuda().expand(-1, -1, 4, -1)
    d = e.contiguous()
    assert torch.equal(pk.qk_norm(e, None)[0], pk.qk_norm(d, None)[0])
    assert torch.equal(pk.qk_norm_backward(e, None, do, None)["dq"], pk.qk_norm_backward(d, None, do, None)["dq"])
    with pytest.raises(pk.OsdnError):
        pk.qk_norm(d, None, q_out=e)


@pytest.mark.gpu
def test_lengths_and_rows_of_zeros():
    """Rows from a length on are neither read nor written nor counted; a row of zeros gives zeros, with
    and without eps, and a finite gradient."""
    import preconditioned_delta_rule_token_b200 as pk
    B, T, H, W = 5, 12, 2, 64
    q, dq = rows(10, B, T, H, W, FP)
    lengths = torch.tensor([0, 1, 12, 40, -2], dtype=torch.int32)
    inside = (torch.arange(T)[None] < lengths[:, None])[..., None, None]
    w = 1 + 0.1 * torch.randn(W, generator=torch.Generator().manual_seed(1))
    how = dict(freqs=ref.plain_freqs(32).cuda(), norm="rms", wq=w.cuda())
    nan_q, nan_d = torch.where(inside, q, float("nan")).cuda(), torch.where(inside, dq, float("nan")).cuda()
    out = torch.full_like(nan_q, 3.0)
    pk.qk_norm(nan_q, None, lengths=lengths.cuda(), q_out=out, **how)
    want = pk.qk_norm(q.cuda(), None, **how)[0]
    assert torch.equal(out, torch.where(inside.cuda(), want, 3.0))
    for eps in (1e-6, 0.0):   # without q_out: zeros there
        own = pk.qk_norm(nan_q, nan_q, lengths=lengths.cuda(), eps=eps, **how)
        assert all(bool((t[~inside.expand_as(q).cuda()] == 0).all()) and bool(torch.isfinite(t).all()) for t in own)
    own = pk.qk_norm(nan_q, nan_q, lengths=lengths.cuda(), q_out=out.fill_(3.0), **how)
    assert bool((own[1][~inside.expand_as(q).cuda()] == 0).all())
    assert torch.equal(out, torch.where(inside.cuda(), want, 3.0))
    got = pk.qk_norm_backward(nan_q, None, nan_d, None, lengths=lengths.cuda(), **how)
    a = ("rms", 1e-6, 1.0, ref.plain_freqs(32), ref.positions_of(B, T), "half", 1.0)
    dx, dw = ref.head_norm_grads(torch.where(inside, q, 1.0), w, torch.where(inside, dq, 0.0), *a)
    ref.close(got["dq"], *dx, 96, "dq")
    assert bool((got["dq"][~inside.expand_as(q).cuda()] == 0).all())
    ref.close(got["dwq"], *dw, B * T * H + 96, "dwq")
    z = torch.zeros(1, 2, 2, 64, device="cuda")
    for eps in (0.0, 1e-6):
        for norm in ("l2", "rms"):
            assert bool((pk.qk_norm(z, None, norm=norm, eps=eps)[0] == 0).all())
            assert bool(torch.isfinite(pk.qk_norm_backward(z, None, z + 1, None, norm=norm, eps=eps)["dq"]).all())
    tiny = torch.full((1, 1, 1, 64), 1e-21, device="cuda")   # squares below fp32's range: as zeros
    assert bool((pk.qk_norm(tiny, None, eps=0.0)[0] == 0).all())
    e = torch.zeros(2, 0, 3, 64, device="cuda")
    assert pk.qk_norm(e, None)[0].shape == e.shape
    assert bool((pk.qk_norm_backward(e, None, e, None, wq=w.cuda())["dwq"] == 0).all())


@pytest.mark.gpu
def test_one_weight_and_given_positions():
    """A weight on q alone, positions from a negative pos0, and the rotation alone with lengths."""
    import preconditioned_delta_rule_token_b200 as pk
    (q, dq), (k, dk) = rows(14, 2, 21, 2, 64, FP), rows(15, 2, 21, 3, 64, FP)
    w = 1 + 0.1 * torch.randn(64, generator=torch.Generator().manual_seed(4))
    fr, pos = ref.plain_freqs(64), ref.positions_of(2, 21, -7)
    how = dict(freqs=fr.cuda(), wq=w.cuda(), pos0=-7, layout="interleaved")
    qo, ko = pk.qk_norm(q.cuda(), k.cuda(), **how)
    g = pk.qk_norm_backward(q.cuda(), k.cuda(), dq.cuda(), dk.cuda(), **how)
    for x, wt, do, out, n in ((q, w, dq, qo, "q"), (k, None, dk, ko, "k")):
        a = ("l2", 1e-6, 1.0, fr, pos, "interleaved", 1.0)
        ref.close(out, *ref.head_norm(x, wt, *a), 32, n)
        dx, dw = ref.head_norm_grads(x, wt, do, *a)
        ref.close(g["d" + n], *dx, 96, "d" + n)
        if wt is not None:
            ref.close(g["dwq"], *dw, 2 * 21 * 2 + 96, "dwq")
    assert g["dwk"] is None
    n = torch.tensor([21, 5], dtype=torch.int32).cuda()
    full, cut = pk.rope(q.cuda(), fr.cuda(), pos0=-7), pk.rope(q.cuda(), fr.cuda(), pos0=-7, lengths=n)
    assert torch.equal(cut[0], full[0]) and torch.equal(cut[1, :5], full[1, :5]) and bool((cut[1, 5:] == 0).all())


@pytest.mark.gpu
def test_against_differences_on_the_device():
    """Directional derivatives of the fp32 forward: over 2 eps = 2^-5 the quotient is off by eps^2 of third
    derivatives and the rounding of the loss over 2 eps: within 1e-2 of the magnitude sum."""
    import preconditioned_delta_rule_token_b200 as pk
    q, dq = (t.cuda() for t in rows(11, 2, 8, 2, 64, FP))
    w = torch.ones(64, device="cuda")
    how = dict(freqs=ref.plain_freqs(64).cuda(), norm="rms")
    got = pk.qk_norm_backward(q, None, dq, None, wq=w, **how)
    g = torch.Generator(device="cuda").manual_seed(3)
    for name, base in (("dq", q), ("dwq", w)):
        v = torch.randn(base.shape, generator=g, device="cuda")
        loss = lambda e: float((pk.qk_norm(q + e * v if name == "dq" else q, None,  # noqa: E731
                                           wq=w + e * v if name == "dwq" else w, **how)[0].double() * dq).sum())
        eps = 2.0 ** -6
        diff, want = (loss(eps) - loss(-eps)) / (2 * eps), got[name].double() * v
        assert abs(diff - float(want.sum())) <= 1e-2 * float(want.abs().sum()), name


@pytest.mark.gpu
def test_repeats_other_streams_and_graphs():
    """Bitwise the same from call to call, on a side stream, and replayed from a graph with new inputs."""
    import preconditioned_delta_rule_token_b200 as pk
    (q, dq), (k, dk) = rows(12, 4, 1500, 4, 64, BF), rows(13, 4, 1500, 2, 64, BF)
    q, dq, k, dk = (t.cuda() for t in (q, dq, k, dk))
    w = torch.ones(64, device="cuda")
    how = dict(freqs=ref.plain_freqs(64).cuda(), norm="rms", wq=w, wk=w, pos0=9)

    def run(q, stream=None):
        g = pk.qk_norm_backward(q, k, dq, dk, stream=stream, **how)
        return list(pk.qk_norm(q, k, stream=stream, **how)) + [g[n] for n in ("dq", "dk", "dwq", "dwk")]

    q2 = torch.randn(q.shape, device="cuda").bfloat16()
    want, want2 = run(q), run(q2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    static = q.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(static)
    for src, exp in ((q2, want2), (q, want)):
        static.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(exp, out))
