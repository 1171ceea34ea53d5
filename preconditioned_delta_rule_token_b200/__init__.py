"""OSDN (Online Scaled DeltaNet) forward, backward and decode on B200 (sm_100a).

The compute lives in ``libosdn.so`` (CUDA kernels behind the C ABI of
``include/osdn.h``); this package is its ctypes binding plus two convenience
wrappers that allocate outputs and workspace with PyTorch:

    out, S, d = forward(q, k, v, beta, r=None, d0=None, S0=None, eta=1e-2)
    grads = backward(q, k, v, beta, dout, r=None, d0=None, S0=None, eta=1e-2)
    o = step(q, k, v, beta, S, d, r=None, eta=1e-2)      # S, d updated in place

Next to them stand what a layer needs around them: the gated linear recurrence
(``recurrence``, ``recurrence_backward``, ``recurrence_step``), the norms of queries and
keys with the position rotation (``qk_norm``, ``qk_norm_backward``) and the rotation
alone (``rope``, ``rope_frequencies``).

All tensors must be CUDA tensors; there is no CPU path.
"""
from __future__ import annotations

import contextlib

import torch

from ._binding import (OSDN_BF16, OSDN_ERR_CUDA, OSDN_ERR_INVALID_ARG, OSDN_ERR_TIMEOUT, OSDN_ERR_UNSUPPORTED,
                       OSDN_FP32, OSDN_OK, LIB_PATH, OsdnError, build, get_last_error, make_params, osdn_fwd,
                       osdn_fwd_chunk, osdn_fwd_scan, osdn_fwd_scan_diag,
                       osdn_fwd_workspace_size, osdn_fwd_segments, osdn_fwd_launches, osdn_params, osdn_set_wait_limit_ns, osdn_step, osdn_step_ex,
                       osdn_fwd_gated, osdn_fwd_chunk_gated, osdn_step_gated,
                       osdn_bwd, osdn_bwd_gated, osdn_bwd_workspace_size, osdn_sync_status,
                       osdn_fwd_host, osdn_fwd_host_buffer_size,
                       osdn_recur_params, osdn_recur_fwd, osdn_recur_bwd, osdn_recur_bwd_workspace_size,
                       osdn_recur_step, osdn_qk_params, osdn_qk_fwd, osdn_qk_bwd, osdn_qk_bwd_workspace_size,
                       osdn_rope, osdn_rope_freqs)
from ._layer import (QkNorm, qk_norm, qk_norm_backward, recurrence, recurrence_backward, recurrence_step, rope,
                     rope_frequencies)

__all__ = ["forward", "backward", "step", "osdn_bwd", "osdn_bwd_gated", "osdn_bwd_workspace_size", "residual_ratio", "osdn_fwd_scan_diag", "osdn_fwd", "osdn_fwd_scan", "osdn_fwd_chunk", "osdn_step", "osdn_fwd_workspace_size", "osdn_fwd_segments", "osdn_fwd_launches", "osdn_sync_status",
           "osdn_set_wait_limit_ns", "osdn_step_ex",
           "osdn_fwd_gated", "osdn_fwd_chunk_gated", "osdn_step_gated", "osdn_fwd_host", "osdn_fwd_host_buffer_size",
           "forward_host", "osdn_params", "make_params", "get_last_error", "OsdnError", "build", "LIB_PATH",
           "OSDN_OK", "OSDN_ERR_INVALID_ARG", "OSDN_ERR_UNSUPPORTED", "OSDN_ERR_CUDA", "OSDN_ERR_TIMEOUT",
           "OSDN_BF16", "OSDN_FP32",
           "recurrence", "recurrence_backward", "recurrence_step", "QkNorm", "qk_norm", "qk_norm_backward", "rope",
           "rope_frequencies", "osdn_recur_params", "osdn_recur_fwd", "osdn_recur_bwd",
           "osdn_recur_bwd_workspace_size", "osdn_recur_step", "osdn_qk_params", "osdn_qk_fwd", "osdn_qk_bwd",
           "osdn_qk_bwd_workspace_size", "osdn_rope", "osdn_rope_freqs"]


def _on(stream):
    """For what a call drops when it returns (workspaces, gradients on the way): allocated on the stream that its
    kernels run on, or the memory could go to the current stream's next allocation while they still use it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _normed(qk, q, k, positions, stream):
    """q and k through qk_norm where its options are given. It also takes fewer key heads than query heads; the
    delta rule wants as many, and its kernels would read q by k's heads."""
    if qk is None:
        if positions is not None:
            raise OsdnError(OSDN_ERR_INVALID_ARG, "positions need qk")
        return q, k
    if q.shape != k.shape:
        raise OsdnError(OSDN_ERR_INVALID_ARG, "the delta rule takes q and k of one shape (got %s and %s)"
                        % (tuple(q.shape), tuple(k.shape)))
    return qk.apply(q, k, positions, stream)


def forward(q, k, v, beta, r=None, d0=None, S0=None, eta=1e-2, chunk=64, workspace=None, stream=None,
            apf_anchor=False, alpha=None, qk=None, positions=None):
    """OSDN forward. q, k [B,T,H,dk]; v [B,T,H,dv]; beta, r [B,T,H] (bf16 or fp32,
    one dtype); d0 [B,H,dk] and S0 [B,H,dv,dk] fp32 or None. apf_anchor: anchored
    APF, the retention pulls d toward d0 instead of 0. alpha [B,T,H] (same dtype): gated OSDN,
    S_t = alpha_t S_{t-1} (I - beta k kw^T) + beta v kw^T (bf16, dk = dv = 128). qk (a QkNorm): q and k
    first go through qk_norm with these options, at `positions` [B,T] int64 (None: 0, 1, ...).
    Returns (out [B,T,H,dv], final_S [B,H,dv,dk] fp32, final_d [B,H,dk] fp32)."""
    q, k = _normed(qk, q, k, positions, stream)
    B, T, H, dk = k.shape
    dv = v.shape[-1]
    p = make_params(B, T, H, dk, dv, k.dtype, eta, chunk, apf_anchor)
    dev = k.device
    out = torch.empty((B, T, H, dv), dtype=k.dtype, device=dev)
    final_S = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    final_d = torch.empty((B, H, dk), dtype=torch.float32, device=dev)
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(osdn_fwd_workspace_size(p), dtype=torch.uint8, device=dev)
    if alpha is None:
        osdn_fwd(p, q, k, v, beta, r, d0, S0, out, final_S, final_d, workspace, stream)
    else:
        osdn_fwd_gated(p, q, k, v, beta, r, alpha, d0, S0, out, final_S, final_d, workspace, stream)
    return out, final_S, final_d


def forward_host(q, k, v, beta, r=None, d0=None, S0=None, eta=1e-2, chunk=64, groups=0, device_buffer=None,
                 stream=None, apf_anchor=False):
    """forward() on HOST tensors (page-locked for overlapped copies): the library copies each group of
    sequences in, runs the forward on it and copies its results back, with the copies of one group
    overlapping the compute of its neighbours (osdn_fwd_host). groups = 0: the library's default.
    Returns host tensors (out, final_S, final_d); the call is asynchronous on `stream`."""
    B, T, H, dk = k.shape
    dv = v.shape[-1]
    p = make_params(B, T, H, dk, dv, k.dtype, eta, chunk, apf_anchor)
    pin = q.is_pinned()
    out = torch.empty((B, T, H, dv), dtype=k.dtype, pin_memory=pin)
    final_S = torch.empty((B, H, dv, dk), dtype=torch.float32, pin_memory=pin)
    final_d = torch.empty((B, H, dk), dtype=torch.float32, pin_memory=pin)
    if device_buffer is None:
        with _on(stream):
            device_buffer = torch.empty(osdn_fwd_host_buffer_size(p, groups), dtype=torch.uint8, device="cuda")
    osdn_fwd_host(p, q, k, v, beta, r, d0, S0, out, final_S, final_d, device_buffer, groups, stream)
    return out, final_S, final_d


def backward(q, k, v, beta, dout, r=None, d0=None, S0=None, dS_final=None, dd_final=None, eta=1e-2, chunk=64,
             workspace=None, stream=None, apf_anchor=False, alpha=None, qk=None, positions=None):
    """Gradients of L = sum(dout * out) + sum(dS_final * final_S) + sum(dd_final * final_d) for the
    forward() with the same inputs (plain or anchored APF; gated OSDN when alpha [B,T,H] is given).
    dout [B,T,H,dv] in the input dtype; dS_final [B,H,dv,dk], dd_final [B,H,dk] fp32 or None (= 0).
    Returns a dict with dq, dk, dv, dbeta, dr (None without r), dalpha (None without alpha) in the
    input dtype and dd0 [B,H,dk], dS0 [B,H,dv,dk] fp32. With qk and positions as in forward(), dq and dk
    are of the q and k before qk_norm (which may be column slices of a projection), and dwq, dwk [dk]
    fp32 of its weights (None without) come too."""
    given = q, k
    q, k = _normed(qk, q, k, positions, stream)
    B, T, H, dk = k.shape
    dv = v.shape[-1]
    p = make_params(B, T, H, dk, dv, k.dtype, eta, chunk, apf_anchor)
    dev, dt = k.device, k.dtype
    with _on(None if qk is None else stream):   # with qk these two are on the way to the raw q's and k's
        g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k)}
    g.update({"dv": torch.empty_like(v),
              "dbeta": torch.empty_like(beta), "dr": None if r is None else torch.empty_like(r),
              "dd0": torch.empty((B, H, dk), dtype=torch.float32, device=dev),
              "dS0": torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)})
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(osdn_bwd_workspace_size(p), dtype=torch.uint8, device=dev)
    if alpha is None:
        osdn_bwd(p, q, k, v, beta, r, d0, S0, dout, dS_final, dd_final, g["dq"], g["dk"], g["dv"], g["dbeta"],
                 g["dr"], g["dd0"], g["dS0"], workspace, stream)
        g["dalpha"] = None
    else:
        g["dalpha"] = torch.empty_like(alpha)
        osdn_bwd_gated(p, q, k, v, beta, r, alpha, d0, S0, dout, dS_final, dd_final, g["dq"], g["dk"], g["dv"],
                       g["dbeta"], g["dr"], g["dalpha"], g["dd0"], g["dS0"], workspace, stream)
    if qk is not None:
        g.update(qk.gradients(*given, g["dq"], g["dk"], positions, stream))
    return g


def residual_ratio(k, beta, r=None, d0=None, eta=1e-2, stream=None, apf_anchor=False):
    """Preconditioner scan with its residual-ratio diagnostic: k [B,T,H,dk]; beta, r [B,T,H];
    d0 [B,H,dk] fp32 (None = ones). Returns rho [B,T,H] fp32 (rho_t = (1 - beta_t <d_t, k_t^2>)^2,
    the factor by which token t's write shrinks its own loss), q_geo [B,H] fp32 (exp of the mean
    log rho over each sequence) and d after the last token [B,H,dk] fp32."""
    B, T, H, dk = k.shape
    p = make_params(B, T, H, dk, dk, k.dtype, eta, apf_anchor=apf_anchor)
    rho = torch.empty((B, T, H), dtype=torch.float32, device=k.device)
    q_geo = torch.empty((B, H), dtype=torch.float32, device=k.device)
    d = torch.empty((B, H, dk), dtype=torch.float32, device=k.device)
    with _on(stream):
        ws = torch.empty(max(osdn_fwd_workspace_size(p), 256), dtype=torch.uint8, device=k.device)
    osdn_fwd_scan_diag(p, k, beta, r, d0, d, rho, q_geo, ws, stream)
    return rho, q_geo, d


def step(q, k, v, beta, S, d, r=None, eta=1e-2, stream=None, d_anchor=None, apf_anchor=False, alpha=None, qk=None,
         positions=None):
    """One decode token for every (b, h): q, k [B,H,dk]; v [B,H,dv]; beta, r [B,H];
    S [B,H,dv,dk] and d [B,H,dk] fp32, updated in place. Anchored APF (apf_anchor, or a
    d_anchor [B,H,dk] fp32 given) pulls d toward d_anchor (ones when None); alpha [B,H] decays S
    first (gated OSDN). qk (a QkNorm): q and k first go through qk_norm at `positions` [B] int64 (None: 0).
    Returns out [B,H,dv]."""
    if qk is None:
        _normed(qk, q, k, positions, stream)
    else:
        q, k = (t.squeeze(1) for t in _normed(qk, q.unsqueeze(1), k.unsqueeze(1),
                                              None if positions is None else positions.unsqueeze(1), stream))
    B, H, dk = k.shape
    dv = v.shape[-1]
    p = make_params(B, 1, H, dk, dv, k.dtype, eta, apf_anchor=apf_anchor or d_anchor is not None)
    out = torch.empty((B, H, dv), dtype=k.dtype, device=k.device)
    if alpha is None:
        osdn_step_ex(p, q, k, v, beta, r, d_anchor, S, d, out, stream)
    else:
        osdn_step_gated(p, q, k, v, beta, r, alpha, d_anchor, S, d, out, stream)
    return out
