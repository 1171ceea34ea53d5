"""What a layer needs next to the delta rule: the gated linear recurrence, the norms of
queries and keys with the position rotation, and the rotation alone.

Wrappers that check shapes, types and devices, allocate the outputs and call the C ABI.
`stream` is a torch.cuda.Stream of the tensors' device (default: that device's current
stream); outputs and workspaces are allocated on it. All tensors must be on one CUDA
device; there is no CPU path. Heads, weights, states and workspaces start on 16 bytes;
x, gate and h of the recurrence start anywhere. An output that is given does not overlap
an input, unless it is said that it may be one.

A decode token's kernels take a few microseconds, so a call does little in Python: the
checks and the parameter block depend on the tensors' layouts (shape, strides, type,
device), the options and the numbers alone and are kept by them, and addresses and stream
go through an extension module (csrc/call.cpp). pos0 is one of the numbers: in a loop over
tokens a positions tensor keeps its block, a pos0 that counts up makes one each time.
"""
from __future__ import annotations

import ctypes
import functools
import operator
from dataclasses import dataclass, fields

import torch

from . import _binding as B
from ._binding import OSDN_BF16, OSDN_ERR_INVALID_ARG, OSDN_ERR_UNSUPPORTED, OSDN_FP32, OsdnError

_DTYPES = {torch.bfloat16: OSDN_BF16, torch.float32: OSDN_FP32}


def _bad(msg, code=OSDN_ERR_INVALID_ARG):
    raise OsdnError(code, msg)


def _scope(dev, stream):
    """Makes `stream` (None: the current one) of device `dev` current for allocations and the launch."""
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        _bad("the stream is of %s, the tensors are on %s" % (stream.device, dev))
    return torch.cuda.stream(stream)


class _Kept(dict):
    """Parameter blocks (and their addresses) by the layouts they were checked for; emptied when it grows past
    1024."""

    def keep(self, key, params):
        if len(self) >= 1024:
            self.clear()
        self[key] = kept = (params, ctypes.addressof(params))
        return kept


class _Calls:
    """The extension module's functions, loaded with the library at the first use."""

    def __getattr__(self, name):
        m = B.call()
        for n in ("layouts", "here", "like", "floats"):
            setattr(self, n, getattr(m, n))
        for n, address in m.fn.items():
            setattr(self, n, functools.partial(getattr(m, n), address))
        return self.__dict__[name]


_C = _Calls()


def _done(rc):
    if rc:
        B._check(rc)


def _choice(name, value, table):
    try:
        return table[value]
    except (KeyError, TypeError):
        _bad("%s is one of %s (got %r)" % (name, ", ".join(table), value))


def _dtype(name, t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        _bad("%s must be bfloat16 or float32 (got %s)" % (name, t.dtype), OSDN_ERR_UNSUPPORTED)
    return code


def _held(dev, name, t, shape, dtype, dense=True):
    """Checks one tensor: on `dev`, of this shape and type, dense where asked."""
    if t is None:
        return
    if t.device != dev or not t.is_cuda:
        _bad("%s is on %s, not on %s (the library has no CPU path)" % (name, t.device, dev))
    if t.shape != shape:
        _bad("%s must be %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        _bad("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if dense and not t.is_contiguous():
        _bad("%s is not contiguous" % name)


def _fits(**sizes):
    """The parameter blocks hold sizes in 32 bits: a larger one would come out as its remainder."""
    for name, n in sizes.items():
        if n >= 1 << 31:
            _bad("%s must be below 2^31 (got %d)" % (name, n))


def _scratch(dev, workspace):
    """Checks a workspace that the caller gave: dense memory of the tensors' device (its size is the library's check)."""
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_cuda:
        _bad("workspace must be a tensor on %s (the library has no CPU path)" % dev)
    if not workspace.is_contiguous():
        _bad("workspace is not contiguous")
    return workspace


def _strides(name, t, n):
    """The first n strides of a token tensor whose last dimension is contiguous (zeros: dense)."""
    if t is None or t.is_contiguous():
        return (0,) * n
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] != 1:
        _bad("the last dimension of %s must be contiguous" % name)
    if not any(st[:n]):
        _bad("%s has strides of 0 in every dimension: expand it into memory" % name)
    return st[:n]


def _rows(name, t, token):
    """Strides over (b, t) of an input of the recurrence; without tokens, one row for all sequences is (0, not 0)."""
    if token:
        return _strides(name, t, 2)
    one = t.shape[0] > 1 and t.stride(0) == 0 and (t.stride(1) == 1 or t.shape[1] == 1)
    return (0, t.shape[1]) if one else (*_strides(name, t, 1), 0)


def _saved(nB, T, D):
    return nB, (T + B.OSDN_RECUR_CHECKPOINT - 1) // B.OSDN_RECUR_CHECKPOINT, D


_RECUR = _Kept()


def _recur_params(x, gate, gate_form, input_scale, named, token=True):
    """Checks a recurrence call and makes its parameter block. named: (name, tensor, kind) with kind "token" (like
    x, any strides), "state" ([B, D] fp32), "lengths" or "saved"."""
    if x.dim() != (3 if token else 2):
        _bad("x is %s (got %s)" % ("[B, T, D]" if token else "[B, D]", tuple(x.shape)))
    if not x.is_cuda:
        _bad("x is on %s (the library has no CPU path)" % x.device)
    dev, code, gcode = x.device, _dtype("x", x), _dtype("gate", gate)
    nB, T, D = x.shape if token else (x.shape[0], 1, x.shape[1])
    _held(dev, "gate", gate, x.shape, gate.dtype, dense=False)
    p = B.osdn_recur_params()
    p.struct_size = ctypes.sizeof(p)
    _fits(B=nB, T=T, D=D)
    p.B, p.T, p.D, p.dtype, p.gate_dtype = nB, T, D, code, gcode
    p.gate_form = _choice("gate_form", gate_form, B.GATE_FORMS)
    p.input_scale = _choice("input_scale", input_scale, B.INPUT_SCALES)
    p.zero_rest = not any(t is not None for name, t, _ in named if name == "h")   # our own outputs
    n = 2 if token else 1
    p.stride_x[:], p.stride_gate[:] = _rows("x", x, token), _rows("gate", gate, token)
    for name, t, kind in named:
        if kind == "token":
            _held(dev, name, t, x.shape, x.dtype, dense=False)
            p.stride_h[:n] = _strides(name, t, n)
        elif kind == "lengths":
            _held(dev, name, t, (nB,), torch.int32)
        else:
            _held(dev, name, t, (nB, D) if kind == "state" else _saved(nB, T, D), torch.float32)
    return p


def recurrence(x, gate, h0=None, lengths=None, gate_form="decay", input_scale="none", checkpoints=False, h=None,
               stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + s_t x_t of every channel.

    x, gate [B,T,D] (x bf16 or fp32; gate of x's type or fp32; the channels contiguous, e.g. column
    slices of one projection). gate_form: a = gate ("decay"), exp(gate) ("log") or sigmoid(gate) ("logit");
    a = 0 starts a new document. input_scale: s = 1 ("none"), 1 - a ("complement") or sqrt(1 - a^2) ("norm").
    h0 [B,D] fp32 or None (zeros). lengths [B] int32 (None: T each): tokens from a sequence's length
    on do not count; their rows of h are zeros (left as they were when `h` is given).
    Returns (h [B,T,D] in x's type, final_h [B,D] fp32), and with checkpoints=True the states
    [B,ceil(T/64),D] fp32 before every 64th token (behind a length: the final state) that
    recurrence_backward takes."""
    key = ("fwd", gate_form, input_scale, _C.layouts(x, gate, h0, lengths, h))
    kept = _RECUR.get(key) or _RECUR.keep(key, _recur_params(
        x, gate, gate_form, input_scale, (("h0", h0, "state"), ("lengths", lengths, "lengths"), ("h", h, "token"))))
    nB, T, D = x.shape
    if stream is not None or not _C.here(x):
        with _scope(x.device, stream):
            return recurrence(x, gate, h0, lengths, gate_form, input_scale, checkpoints, h)
    if h is None:
        h = _C.like(x)
    final_h = _C.floats(x, nB, D)
    marks = _C.floats(x, *_saved(nB, T, D)) if checkpoints else None
    _done(_C.recur_fwd(kept[1], x, gate, h0, lengths, h, final_h, marks))
    return (h, final_h, marks) if checkpoints else (h, final_h)


def recurrence_backward(x, gate, dh, h0=None, dfinal_h=None, lengths=None, checkpoints=None, gate_form="decay",
                        input_scale="none", workspace=None, stream=None):
    """Gradients of L = sum(dh * h) + sum(dfinal_h * final_h) for the recurrence() of the same inputs.

    dh [B,T,D] in x's type (the channels contiguous); dfinal_h [B,D] fp32 or None (= 0). checkpoints: the states that
    recurrence(..., checkpoints=True) returned for the same inputs; None runs the forward again for them.
    Returns a dict with dx (x's type), dgate (the gate's type; with respect to the gate as given) and
    dh0 [B,D] fp32. Rows from a sequence's length on are zeros."""
    key = ("bwd", gate_form, input_scale, _C.layouts(x, gate, dh, h0, dfinal_h, lengths, checkpoints))
    kept = _RECUR.get(key) or _RECUR.keep(key, _recur_params(
        x, gate, gate_form, input_scale,
        (("h0", h0, "state"), ("lengths", lengths, "lengths"), ("dh", dh, "token"), ("dfinal_h", dfinal_h, "state"),
         ("checkpoints", checkpoints, "saved"))))
    if stream is not None or not _C.here(x):
        with _scope(x.device, stream):
            return recurrence_backward(x, gate, dh, h0, dfinal_h, lengths, checkpoints, gate_form, input_scale,
                                       workspace)
    g = {"dx": _C.like(x), "dgate": _C.like(gate),
         "dh0": _C.floats(x, x.shape[0], x.shape[2])}
    if workspace is not None:
        _scratch(x.device, workspace)
    elif checkpoints is None:
        workspace = torch.empty(B.osdn_recur_bwd_workspace_size(kept[0]), dtype=torch.uint8, device=x.device)
    _done(_C.recur_bwd(kept[1], x, gate, h0, lengths, dh, dfinal_h, checkpoints, g["dx"], g["dgate"], g["dh0"],
                       workspace))
    return g


def recurrence_step(x, gate, state, gate_form="decay", input_scale="none", out=None, stream=None):
    """One decode token of the recurrence: x, gate [B,D] (or one row of them expanded over the batch); state [B,D]
    fp32, updated in place.
    Returns the new state in x's type [B,D] (`out` if given)."""
    key = ("step", gate_form, input_scale, _C.layouts(x, gate, state, out))
    kept = _RECUR.get(key) or _RECUR.keep(key, _recur_params(
        x, gate, gate_form, input_scale, (("state", state, "state"), ("out", out, "token")), token=False))
    if stream is not None or not _C.here(x):
        with _scope(x.device, stream):
            return recurrence_step(x, gate, state, gate_form, input_scale, out)
    if out is None:
        out = _C.like(x)
    _done(_C.recur_step(kept[1], x, gate, state, out))
    return out


_HEADS = _Kept()


def _numbers(eps, amplitude, scale_q, scale_k, pos0):
    """The numbers of a call by value: a block is kept by them alone, for a tensor in their place (a learned scale) is
    known by its identity while its value changes. It meets no kept block, and is converted on every call."""
    try:
        return float(eps), float(amplitude), float(scale_q), float(scale_k), operator.index(pos0)
    except (TypeError, ValueError, RuntimeError):
        _bad("eps, amplitude and the scales are numbers, pos0 is an integer (got %s)" %
             ", ".join(type(v).__name__ for v in (eps, amplitude, scale_q, scale_k, pos0)))


def _heads_params(q, k, freqs, positions, lengths, norm, layout, wq, wk, out_q, out_k, numbers, names):
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        _bad("%s [B, T, H, width]" % ("%s and %s are" % names[:2] if names[1] else "%s is" % names[0]))
    if not q.is_cuda:
        _bad("%s is on %s (the library has no CPU path)" % (names[0], q.device))
    (nB, T, Hq, width), dev = q.shape, q.device
    Hk = 0 if k is None else k.shape[2]
    p = B.osdn_qk_params()
    p.struct_size = ctypes.sizeof(p)
    _fits(B=nB, T=T, Hq=Hq, Hk=Hk, width=width, rot_dim=0 if freqs is None else 2 * freqs.numel())
    if abs(numbers[-1]) > 1 << 53:
        _bad("pos0 must lie within +-2^53 (got %d)" % numbers[-1])
    p.B, p.T, p.Hq, p.Hk, p.width, p.dtype = nB, T, Hq, Hk, width, _dtype(names[0], q)
    p.norm, p.layout = _choice("norm", norm, B.NORMS), _choice("layout", layout, B.ROPE_LAYOUTS)
    p.eps, p.amplitude, p.scale_q, p.scale_k, p.pos0 = numbers
    p.zero_rest = names[2].startswith("d") or (out_q is None and out_k is None)   # our own outputs
    if k is not None:
        _held(dev, names[1], k, (nB, T, Hk, width), q.dtype, dense=False)
        _held(dev, names[3], out_k, k.shape, q.dtype, dense=False)
        p.stride_k[:], p.stride_out_k[:] = _strides(names[1], k, 3), _strides(names[3], out_k, 3)
    _held(dev, names[2], out_q, q.shape, q.dtype, dense=False)
    p.stride_q[:], p.stride_out_q[:] = _strides(names[0], q, 3), _strides(names[2], out_q, 3)
    _held(dev, "positions", positions, (nB, T), torch.int64)
    _held(dev, "lengths", lengths, (nB,), torch.int32)
    _held(dev, "wq", wq, (width,), torch.float32)
    _held(dev, "wk", wk, (width,), torch.float32)
    if freqs is not None:
        _held(dev, "freqs", freqs, (freqs.numel(),), torch.float64)
        p.rot_dim = 2 * freqs.numel()
    return p


def qk_norm(q, k, freqs=None, positions=None, norm="l2", eps=1e-6, wq=None, wk=None, layout="half", amplitude=1.0,
            scale_q=1.0, scale_k=1.0, pos0=0, lengths=None, q_out=None, k_out=None, stream=None):
    """Norm of every query and key head, then the position rotation, in one pass.

    q [B,T,Hq,width], k [B,T,Hk,width] or None (bf16 or fp32; column slices of a fused projection are
    read in place). norm: "l2" (x / sqrt(sum x^2 + eps), as the delta rule wants its keys), "rms"
    (x / sqrt(mean x^2 + eps)) or "none"; wq, wk [width] fp32 multiply after it, scale_q and scale_k too.
    freqs [rot/2] fp64 (rope_frequencies; None: no rotation) turns the first rot features: pairs
    (i, i + rot/2) for layout "half" (rot a multiple of 8), (2i, 2i+1) for "interleaved". positions
    [B,T] int64 (None: pos0 + t). lengths [B] int32: tokens from a sequence's length on give zeros
    (rows of a given q_out, k_out stay as they were). q_out may be q, k_out may be k.
    Returns (q_out, k_out)."""
    layouts = _C.layouts(q, k, freqs, positions, lengths, wq, wk, q_out, k_out)
    kept = _HEADS.get((norm, layout, (eps, amplitude, scale_q, scale_k, pos0), layouts))
    if kept is None:
        numbers = _numbers(eps, amplitude, scale_q, scale_k, pos0)
        kept = _HEADS.keep((norm, layout, numbers, layouts), _heads_params(
            q, k, freqs, positions, lengths, norm, layout, wq, wk, q_out, k_out, numbers, ("q", "k", "q_out", "k_out")))
    if stream is not None or not _C.here(q):
        with _scope(q.device, stream):
            return qk_norm(q, k, freqs, positions, norm, eps, wq, wk, layout, amplitude, scale_q, scale_k, pos0, lengths,
                           q_out, k_out)
    both = lengths is None or (q_out is None and k_out is None)
    if q_out is None:
        q_out = _C.like(q) if both else torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    if k is not None and k_out is None:
        k_out = _C.like(k) if both else torch.zeros(k.shape, dtype=k.dtype, device=k.device)
    _done(_C.qk_fwd(kept[1], q, k, wq, wk, positions, freqs, lengths, q_out, k_out))
    return q_out, k_out


def qk_norm_backward(q, k, dq_out, dk_out, freqs=None, positions=None, norm="l2", eps=1e-6, wq=None, wk=None,
                     layout="half", amplitude=1.0, scale_q=1.0, scale_k=1.0, pos0=0, lengths=None, workspace=None,
                     stream=None):
    """Gradients of L = sum(dq_out * q_out) + sum(dk_out * k_out) for the qk_norm() of the same inputs.
    Returns a dict with dq, dk (the inputs' type; zeros from a sequence's length on) and dwq, dwk
    [width] fp32 (None without the weight)."""
    if (k is None) != (dk_out is None):
        _bad("k and dk_out go together")
    layouts = _C.layouts(q, k, freqs, positions, lengths, wq, wk, dq_out, dk_out)
    kept = _HEADS.get(("bwd", norm, layout, (eps, amplitude, scale_q, scale_k, pos0), layouts))
    if kept is None:
        numbers = _numbers(eps, amplitude, scale_q, scale_k, pos0)
        kept = _HEADS.keep(("bwd", norm, layout, numbers, layouts), _heads_params(
            q, k, freqs, positions, lengths, norm, layout, wq, wk, dq_out, dk_out, numbers,
            ("q", "k", "dq_out", "dk_out")))
    if stream is not None or not _C.here(q):
        with _scope(q.device, stream):
            return qk_norm_backward(q, k, dq_out, dk_out, freqs, positions, norm, eps, wq, wk, layout, amplitude, scale_q,
                                    scale_k, pos0, lengths, workspace)
    g = {"dq": _C.like(q), "dk": None if k is None else _C.like(k),
         "dwq": None if wq is None else _C.like(wq),
         "dwk": None if wk is None or k is None else _C.like(wk)}
    if g["dwk"] is not None and not k.shape[2]:   # no key heads: the library takes k, and so wk, as not given
        g["dwk"].zero_()
    if workspace is not None:
        _scratch(q.device, workspace)
    elif g["dwq"] is not None or g["dwk"] is not None:
        workspace = torch.empty(B.osdn_qk_bwd_workspace_size(kept[0]), dtype=torch.uint8, device=q.device)
    _done(_C.qk_bwd(kept[1], q, k, wq, wk, positions, freqs, lengths, dq_out, dk_out, g["dq"], g["dk"], g["dwq"],
                    g["dwk"], workspace))
    return g


@dataclass(frozen=True)
class QkNorm:
    """Options of qk_norm for forward(), backward() and step(), which then take q and k before it: the delta
    rule wants keys of unit length."""
    norm: str = "l2"
    eps: float = 1e-6
    wq: torch.Tensor | None = None
    wk: torch.Tensor | None = None
    freqs: torch.Tensor | None = None
    layout: str = "half"
    amplitude: float = 1.0
    scale_q: float = 1.0
    scale_k: float = 1.0

    def _options(self):
        return {f.name: getattr(self, f.name) for f in fields(self)}

    def apply(self, q, k, positions=None, stream=None):
        return qk_norm(q, k, positions=positions, stream=stream, **self._options())

    def gradients(self, q, k, dq_out, dk_out, positions=None, stream=None):
        return qk_norm_backward(q, k, dq_out, dk_out, positions=positions, stream=stream, **self._options())


def rope(x, freqs, positions=None, layout="half", amplitude=1.0, scale=1.0, pos0=0, inverse=False, lengths=None,
         out=None, stream=None):
    """The position rotation alone on x [B,T,H,width]: see qk_norm for freqs, positions, layout and lengths.
    inverse=True turns back with the same amplitude: it takes the gradient of the result to that of x.
    `out` may be x. Returns the rotated tensor."""
    layouts = _C.layouts(x, freqs, positions, lengths, out)
    kept = _HEADS.get(("rope", layout, (0.0, amplitude, scale, 1.0, pos0), layouts))
    if kept is None:
        if freqs is None:
            _bad("freqs is needed")
        numbers = _numbers(0.0, amplitude, scale, 1.0, pos0)
        kept = _HEADS.keep(("rope", layout, numbers, layouts), _heads_params(
            x, None, freqs, positions, lengths, "none", layout, None, None, out, None, numbers,
            ("x", None, "out", None)))
    if stream is not None or not _C.here(x):
        with _scope(x.device, stream):
            return rope(x, freqs, positions, layout, amplitude, scale, pos0, inverse, lengths, out)
    if out is None:
        out = _C.like(x)
    _done(_C.rope(kept[1], x, positions, freqs, lengths, out, 1 if inverse else 0))
    return out


def rope_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_length=0, low_turns=1.0,
                     high_turns=None, device="cuda"):
    """Frequencies of the rotation of rot_dim features as a fp64 tensor [rot_dim/2], and its amplitude.

    scaling, for contexts `factor` times longer than original_length: "none"; "linear" (all divided by
    factor); "ntk" (a larger base); "yarn" (pairs with more than high_turns turns over original_length
    kept, fewer than low_turns divided, a ramp over the pairs between; amplitude 0.1 ln(factor) + 1);
    "wavelength" (the ramp over the number of turns). high_turns defaults to 32 ("yarn") or 4."""
    if high_turns is None:
        high_turns = 32.0 if scaling == "yarn" else 4.0
    f, amplitude = B.osdn_rope_freqs(int(rot_dim), float(base), _choice("scaling", scaling, B.ROPE_SCALINGS),
                                     float(factor), int(original_length), float(low_turns), float(high_turns))
    return torch.tensor(f, dtype=torch.float64, device=device), amplitude
