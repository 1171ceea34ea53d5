"""ctypes binding of libosdn.so (argument marshalling only).

Every arithmetic step runs in the library's CUDA kernels; this module checks
tensors, builds the ``osdn_params`` block and passes raw device pointers and
the current CUDA stream. It raises if the library is missing or the tensors
are not on a CUDA device: there is no CPU path.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import subprocess
import sysconfig

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
_CSRC = os.path.join(_PKG, "csrc")
_INCLUDE = os.path.join(_ROOT, "include")
LIB_PATH = os.path.join(_PKG, "libosdn.so")

OSDN_OK, OSDN_ERR_INVALID_ARG, OSDN_ERR_UNSUPPORTED, OSDN_ERR_CUDA, OSDN_ERR_TIMEOUT = range(5)
OSDN_BF16, OSDN_FP32 = 0, 1
OSDN_NOALLOC_SCRATCH_BYTES = 32 << 20
OSDN_RECUR_CHECKPOINT = 64
GATE_FORMS = {"decay": 0, "log": 1, "logit": 2}
INPUT_SCALES = {"none": 0, "complement": 1, "norm": 2}
NORMS = {"none": 0, "l2": 1, "rms": 2}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4}

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "-cudart", "static", "--expt-relaxed-constexpr"]


class osdn_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("B", ctypes.c_int32), ("T", ctypes.c_int32),
                ("H", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("chunk", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eta", ctypes.c_float),
                ("apf_anchor", ctypes.c_int32), ("stride_q", ctypes.c_int64 * 3), ("stride_k", ctypes.c_int64 * 3),
                ("stride_v", ctypes.c_int64 * 3), ("stride_o", ctypes.c_int64 * 3)]


class osdn_recur_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("B", ctypes.c_int32), ("T", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32),
                ("gate_form", ctypes.c_int32), ("input_scale", ctypes.c_int32), ("zero_rest", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("stride_x", ctypes.c_int64 * 2),
                ("stride_gate", ctypes.c_int64 * 2), ("stride_h", ctypes.c_int64 * 2)]


class osdn_qk_params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("B", ctypes.c_int32), ("T", ctypes.c_int32),
                ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("layout", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("eps", ctypes.c_float), ("amplitude", ctypes.c_float), ("scale_q", ctypes.c_float),
                ("scale_k", ctypes.c_float), ("zero_rest", ctypes.c_int32), ("reserved", ctypes.c_int32), ("pos0", ctypes.c_int64), ("stride_q", ctypes.c_int64 * 3),
                ("stride_k", ctypes.c_int64 * 3), ("stride_out_q", ctypes.c_int64 * 3),
                ("stride_out_k", ctypes.c_int64 * 3)]


class OsdnError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("osdn error %d: %s" % (code, msg))
        self.code = code


def _sources():
    return sorted(os.path.join(_CSRC, f) for f in os.listdir(_CSRC) if f.endswith((".cu", ".cuh")))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libosdn.so in-tree for sm_100a with nvcc."""
    deps = _sources() + [os.path.join(_INCLUDE, "osdn.h")]
    if not force and os.path.exists(LIB_PATH):
        if os.path.getmtime(LIB_PATH) >= max(os.path.getmtime(p) for p in deps):
            return LIB_PATH
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = ["nvcc"] + NVCC_FLAGS + ["-I", _INCLUDE, "-I", _CSRC, "-o", tmp, os.path.join(_CSRC, "osdn_api.cu")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.check_call(cmd)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build_if_missing() -> str:
    return build(force=False)


# The extension module is compiled against torch's C++ headers: one file for each torch.
CALL_PATH = os.path.join(_PKG, "_call." + torch.__version__ + sysconfig.get_config_var("EXT_SUFFIX"))


def build_call(force: bool = False) -> str:
    """Compile the extension module that the layer's wrappers call through (csrc/call.cpp), in-tree with g++."""
    src = os.path.join(_CSRC, "call.cpp")
    if not force and os.path.exists(CALL_PATH) and os.path.getmtime(CALL_PATH) >= os.path.getmtime(src):
        return CALL_PATH
    home = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_path("include"), os.path.join(cuda, "include")]
    libs, tmp = os.path.join(home, "lib"), CALL_PATH + ".tmp%d" % os.getpid()
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
                           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI] +
                          ["-I" + d for d in include] + ["-o", tmp, src, "-L" + libs, "-ltorch_python", "-ltorch",
                                                         "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + libs])
    os.replace(tmp, CALL_PATH)
    return CALL_PATH


_call = None


def call():
    """The extension module, and in it the addresses of the library's functions as `fn` (built if missing)."""
    global _call
    if _call is None:
        L = lib()
        try:
            build_call(force=False)
        except (OSError, subprocess.CalledProcessError) as exc:
            if not os.path.exists(CALL_PATH):
                raise OsdnError(OSDN_ERR_UNSUPPORTED, "_call is not built and g++ failed: %s" % exc)
        name = __package__ + "._call"
        spec = importlib.util.spec_from_file_location(
            name, CALL_PATH, loader=importlib.machinery.ExtensionFileLoader(name, CALL_PATH))
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.fn = {n: ctypes.cast(getattr(L, "osdn_" + n), ctypes.c_void_p).value
                for n in ("recur_fwd", "recur_bwd", "recur_step", "qk_fwd", "qk_bwd", "rope")}
        _call = m
    return _call


_lib = None


def lib():
    """The loaded library (raises if it was never built)."""
    global _lib
    if _lib is None:
        try:
            build(force=False)          # rebuild in-tree when a source is newer than the library
        except (OSError, subprocess.CalledProcessError) as exc:
            if not os.path.exists(LIB_PATH):
                raise OsdnError(OSDN_ERR_UNSUPPORTED, "libosdn.so is not built and nvcc failed: %s" % exc)
        L = ctypes.CDLL(LIB_PATH)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        P = ctypes.POINTER(osdn_params)
        L.osdn_fwd_workspace_size.argtypes = [P, ctypes.POINTER(sz)]
        L.osdn_fwd_workspace_size.restype = ctypes.c_int
        L.osdn_fwd_segments.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
        L.osdn_fwd_segments.restype = ctypes.c_int
        L.osdn_fwd_launches.argtypes = [P, ctypes.POINTER(ctypes.c_int)]
        L.osdn_fwd_launches.restype = ctypes.c_int
        L.osdn_fwd.argtypes = [P] + [vp] * 10 + [vp, sz, vp]
        L.osdn_fwd.restype = ctypes.c_int
        L.osdn_fwd_scan.argtypes = [P] + [vp] * 5 + [vp, sz, vp]
        L.osdn_fwd_scan.restype = ctypes.c_int
        L.osdn_fwd_scan_diag.argtypes = [P] + [vp] * 7 + [vp, sz, vp]
        L.osdn_fwd_scan_diag.restype = ctypes.c_int
        L.osdn_fwd_chunk.argtypes = [P] + [vp] * 7 + [vp, sz, vp]
        L.osdn_fwd_chunk.restype = ctypes.c_int
        L.osdn_fwd_noalloc.argtypes = [P] + [vp] * 10 + [vp]
        L.osdn_fwd_noalloc.restype = ctypes.c_int
        L.osdn_step.argtypes = [P] + [vp] * 8 + [vp]
        L.osdn_step.restype = ctypes.c_int
        L.osdn_step_ex.argtypes = [P] + [vp] * 9 + [vp]
        L.osdn_step_ex.restype = ctypes.c_int
        L.osdn_step_gated.argtypes = [P] + [vp] * 10 + [vp]
        L.osdn_step_gated.restype = ctypes.c_int
        L.osdn_fwd_gated.argtypes = [P] + [vp] * 11 + [vp, sz, vp]
        L.osdn_fwd_gated.restype = ctypes.c_int
        L.osdn_fwd_chunk_gated.argtypes = [P] + [vp] * 8 + [vp, sz, vp]
        L.osdn_fwd_chunk_gated.restype = ctypes.c_int
        L.osdn_fwd_host_buffer_size.argtypes = [P, ctypes.c_int, ctypes.POINTER(sz)]
        L.osdn_fwd_host_buffer_size.restype = ctypes.c_int
        L.osdn_fwd_host.argtypes = [P] + [vp] * 10 + [vp, sz, ctypes.c_int, vp]
        L.osdn_fwd_host.restype = ctypes.c_int
        L.osdn_bwd_workspace_size.argtypes = [P, ctypes.POINTER(sz)]
        L.osdn_bwd_workspace_size.restype = ctypes.c_int
        L.osdn_bwd.argtypes = [P] + [vp] * 17 + [vp, sz, vp]
        L.osdn_bwd.restype = ctypes.c_int
        L.osdn_bwd_gated.argtypes = [P] + [vp] * 20 + [sz, vp]
        L.osdn_bwd_gated.restype = ctypes.c_int
        R, Q = ctypes.POINTER(osdn_recur_params), ctypes.POINTER(osdn_qk_params)
        psz, dbl, pdbl = ctypes.POINTER(sz), ctypes.c_double, ctypes.POINTER(ctypes.c_double)
        for name, args in (("osdn_recur_fwd", [R] + [vp] * 8), ("osdn_recur_bwd_workspace_size", [R, psz]),
                           ("osdn_recur_bwd", [R] + [vp] * 11 + [sz, vp]), ("osdn_recur_step", [R] + [vp] * 5),
                           ("osdn_qk_fwd", [Q] + [vp] * 10), ("osdn_qk_bwd_workspace_size", [Q, psz]),
                           ("osdn_qk_bwd", [Q] + [vp] * 14 + [sz, vp]),
                           ("osdn_rope", [Q] + [vp] * 5 + [ctypes.c_int, vp]),
                           ("osdn_rope_freqs", [ctypes.c_int32, dbl, ctypes.c_int32, dbl, ctypes.c_int64, dbl, dbl,
                                                pdbl, pdbl])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_int
        L.osdn_sync_status.argtypes = [vp]
        L.osdn_sync_status.restype = ctypes.c_int
        L.osdn_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.osdn_set_wait_limit_ns.restype = None
        L.osdn_get_last_error.argtypes = []
        L.osdn_get_last_error.restype = ctypes.c_char_p
        L.osdn_abi_version.argtypes = []
        L.osdn_abi_version.restype = ctypes.c_int
        _lib = L
    return _lib


def get_last_error() -> str:
    return lib().osdn_get_last_error().decode()


def _check(rc):
    if rc != OSDN_OK:
        raise OsdnError(rc, get_last_error())


def make_params(B, T, H, dk, dv, dtype, eta, chunk=64, apf_anchor=False) -> osdn_params:
    p = osdn_params()
    p.struct_size = ctypes.sizeof(osdn_params)
    p.B, p.T, p.H, p.dk, p.dv, p.chunk = int(B), int(T), int(H), int(dk), int(dv), int(chunk)
    p.dtype = OSDN_BF16 if dtype == torch.bfloat16 else OSDN_FP32
    p.eta = float(eta)
    p.apf_anchor = 1 if apf_anchor else 0
    return p


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise OsdnError(OSDN_ERR_INVALID_ARG, "tensor is not on a CUDA device (the library has no CPU path)")
    if not t.is_contiguous():
        raise OsdnError(OSDN_ERR_INVALID_ARG, "tensor is not contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _ptr_tok(t):
    """Pointer of a token tensor [B, T, H, width] that may be a strided view (last dimension contiguous);
    its other strides go into the parameter block (_set_strides)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise OsdnError(OSDN_ERR_INVALID_ARG, "tensor is not on a CUDA device (the library has no CPU path)")
    if t.dim() != 4 or (t.numel() > 0 and t.stride(-1) != 1):
        raise OsdnError(OSDN_ERR_INVALID_ARG, "token tensors are [B, T, H, width] with the last dimension contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _host_ptr(t):
    """Pointer of a dense host tensor (page-locked memory lets its copies overlap; pageable works too)."""
    if t is None:
        return None
    if t.is_cuda:
        raise OsdnError(OSDN_ERR_INVALID_ARG, "osdn_fwd_host takes host tensors (the device data lives in device_buffer)")
    if not t.is_contiguous():
        raise OsdnError(OSDN_ERR_INVALID_ARG, "tensor is not contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _set_strides(params, q=None, k=None, v=None, out=None):
    """Copy the (b, t, h) element strides of q, k, v, out into params (zeros: dense)."""
    for name, t in (("stride_q", q), ("stride_k", k), ("stride_v", v), ("stride_o", out)):
        dense = t is None or t.is_contiguous()
        getattr(params, name)[:] = (0, 0, 0) if dense else (t.stride(0), t.stride(1), t.stride(2))
    return params


def _current_stream(device_index):
    """Handle of the current stream of a device (what torch.cuda.current_stream().cuda_stream gives, without
    making a Stream object: 3 us less a call)."""
    return torch._C._cuda_getCurrentRawStream(device_index)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def osdn_fwd_workspace_size(params: osdn_params) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().osdn_fwd_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def osdn_fwd_launches(params: osdn_params) -> int:
    """Kernel launches of one osdn_fwd call with these parameters."""
    n = ctypes.c_int(0)
    _check(lib().osdn_fwd_launches(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def osdn_fwd_segments(params: osdn_params) -> int:
    """Segments per sequence that phase 2 splits into (1: none)."""
    n = ctypes.c_int(0)
    _check(lib().osdn_fwd_segments(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def osdn_fwd(params, q, k, v, beta, r, d0, S0, out, final_S, final_d, workspace, stream=None):
    """Raw C-ABI call: every tensor preallocated by the caller (device memory)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _set_strides(params, q, k, v, out)
    _check(lib().osdn_fwd(ctypes.byref(params), _ptr_tok(q), _ptr_tok(k), _ptr_tok(v), _ptr(beta), _ptr(r), _ptr(d0),
                          _ptr(S0), _ptr_tok(out), _ptr(final_S), _ptr(final_d), _ptr(workspace), ctypes.c_size_t(ws_bytes),
                          _stream(stream)))


def _ws_bytes(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def osdn_fwd_host_buffer_size(params: osdn_params, groups: int = 0) -> int:
    """Bytes of the device buffer osdn_fwd_host needs for these parameters and group count."""
    n = ctypes.c_size_t(0)
    _check(lib().osdn_fwd_host_buffer_size(ctypes.byref(params), ctypes.c_int(int(groups)), ctypes.byref(n)))
    return n.value


def osdn_fwd_host(params, q, k, v, beta, r, d0, S0, out, final_S, final_d, device_buffer, groups=0, stream=None):
    """Raw C-ABI call: inputs and outputs are dense HOST tensors, device_buffer a CUDA tensor of at
    least osdn_fwd_host_buffer_size bytes."""
    _check(lib().osdn_fwd_host(ctypes.byref(params), _host_ptr(q), _host_ptr(k), _host_ptr(v), _host_ptr(beta),
                               _host_ptr(r), _host_ptr(d0), _host_ptr(S0), _host_ptr(out), _host_ptr(final_S),
                               _host_ptr(final_d), _ptr(device_buffer), ctypes.c_size_t(_ws_bytes(device_buffer)),
                               ctypes.c_int(int(groups)), _stream(stream)))


def osdn_fwd_scan(params, k, beta, r, d0, final_d, workspace, stream=None):
    """Raw C-ABI call of phase 1 (preconditioner scan into the workspace)."""
    _set_strides(params, k=k)
    _check(lib().osdn_fwd_scan(ctypes.byref(params), _ptr_tok(k), _ptr(beta), _ptr(r), _ptr(d0), _ptr(final_d),
                               _ptr(workspace), ctypes.c_size_t(_ws_bytes(workspace)), _stream(stream)))


def osdn_fwd_scan_diag(params, k, beta, r, d0, final_d, rho, q_geo, workspace, stream=None):
    """Raw C-ABI call of phase 1 with the residual-ratio diagnostic (rho, q_geo nullable)."""
    _set_strides(params, k=k)
    _check(lib().osdn_fwd_scan_diag(ctypes.byref(params), _ptr_tok(k), _ptr(beta), _ptr(r), _ptr(d0), _ptr(final_d),
                                    _ptr(rho), _ptr(q_geo), _ptr(workspace), ctypes.c_size_t(_ws_bytes(workspace)),
                                    _stream(stream)))


def osdn_fwd_chunk(params, q, k, v, beta, S0, out, final_S, workspace, stream=None):
    """Raw C-ABI call of phase 2 (chunked delta rule reading the workspace)."""
    _set_strides(params, q, k, v, out)
    _check(lib().osdn_fwd_chunk(ctypes.byref(params), _ptr_tok(q), _ptr_tok(k), _ptr_tok(v), _ptr(beta), _ptr(S0),
                                _ptr_tok(out),
                                _ptr(final_S), _ptr(workspace), ctypes.c_size_t(_ws_bytes(workspace)),
                                _stream(stream)))


def osdn_fwd_noalloc(params, q, k, v, beta, r, d0, S0, out, final_S, final_d, stream=None):
    """Raw C-ABI call of the forward that takes no workspace: the library uses
    its own fixed scratch array (see OSDN_NOALLOC_SCRATCH_BYTES in osdn.h)."""
    _set_strides(params, q, k, v, out)
    _check(lib().osdn_fwd_noalloc(ctypes.byref(params), _ptr_tok(q), _ptr_tok(k), _ptr_tok(v), _ptr(beta), _ptr(r),
                                  _ptr(d0), _ptr(S0), _ptr_tok(out), _ptr(final_S), _ptr(final_d), _stream(stream)))


def osdn_step(params, q, k, v, beta, r, S, d, out, stream=None):
    """Raw C-ABI call: one decode token for every (b, h); S and d updated in place."""
    _check(lib().osdn_step(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(r), _ptr(S), _ptr(d),
                           _ptr(out), _stream(stream)))


def osdn_step_ex(params, q, k, v, beta, r, d_anchor, S, d, out, stream=None):
    """Raw C-ABI call: osdn_step with anchored APF toward d_anchor when params.apf_anchor is set."""
    _check(lib().osdn_step_ex(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(r), _ptr(d_anchor),
                              _ptr(S), _ptr(d), _ptr(out), _stream(stream)))


def osdn_fwd_gated(params, q, k, v, beta, r, alpha, d0, S0, out, final_S, final_d, workspace, stream=None):
    """Raw C-ABI call of the gated forward (alpha decay of the state)."""
    _set_strides(params, q, k, v, out)
    _check(lib().osdn_fwd_gated(ctypes.byref(params), _ptr_tok(q), _ptr_tok(k), _ptr_tok(v), _ptr(beta), _ptr(r),
                                _ptr(alpha), _ptr(d0), _ptr(S0), _ptr_tok(out), _ptr(final_S), _ptr(final_d),
                                _ptr(workspace),
                                ctypes.c_size_t(_ws_bytes(workspace)), _stream(stream)))


def osdn_fwd_chunk_gated(params, q, k, v, beta, alpha, S0, out, final_S, workspace, stream=None):
    """Raw C-ABI call of phase 2 of the gated forward."""
    _set_strides(params, q, k, v, out)
    _check(lib().osdn_fwd_chunk_gated(ctypes.byref(params), _ptr_tok(q), _ptr_tok(k), _ptr_tok(v), _ptr(beta),
                                      _ptr(alpha), _ptr(S0), _ptr_tok(out), _ptr(final_S), _ptr(workspace),
                                      ctypes.c_size_t(_ws_bytes(workspace)), _stream(stream)))


def osdn_step_gated(params, q, k, v, beta, r, alpha, d_anchor, S, d, out, stream=None):
    """Raw C-ABI call: one gated decode token for every (b, h)."""
    _check(lib().osdn_step_gated(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(r), _ptr(alpha),
                                 _ptr(d_anchor), _ptr(S), _ptr(d), _ptr(out), _stream(stream)))


def osdn_bwd_workspace_size(params: osdn_params) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().osdn_bwd_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def osdn_bwd(params, q, k, v, beta, r, d0, S0, dout, dS_final, dd_final, dq, dk, dv, dbeta, dr, dd0, dS0, workspace,
             stream=None):
    """Raw C-ABI call of the backward: every tensor preallocated by the caller (device memory)."""
    _check(lib().osdn_bwd(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(r), _ptr(d0), _ptr(S0),
                          _ptr(dout), _ptr(dS_final), _ptr(dd_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta),
                          _ptr(dr), _ptr(dd0), _ptr(dS0), _ptr(workspace), ctypes.c_size_t(_ws_bytes(workspace)),
                          _stream(stream)))


def osdn_bwd_gated(params, q, k, v, beta, r, alpha, d0, S0, dout, dS_final, dd_final, dq, dk, dv, dbeta, dr, dalpha,
                   dd0, dS0, workspace, stream=None):
    """Raw C-ABI call of the gated backward: as osdn_bwd plus alpha [B,T,H] and dalpha [B,T,H]."""
    _check(lib().osdn_bwd_gated(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(r), _ptr(alpha),
                                _ptr(d0), _ptr(S0), _ptr(dout), _ptr(dS_final), _ptr(dd_final), _ptr(dq), _ptr(dk),
                                _ptr(dv), _ptr(dbeta), _ptr(dr), _ptr(dalpha), _ptr(dd0), _ptr(dS0), _ptr(workspace),
                                ctypes.c_size_t(_ws_bytes(workspace)), _stream(stream)))


def _ptr_rows(t):
    """Address of a token tensor whose last dimension is contiguous; its other strides are in the parameter block."""
    if t is None:
        return None
    if not t.is_cuda:
        raise OsdnError(OSDN_ERR_INVALID_ARG, "tensor is not on a CUDA device (the library has no CPU path)")
    if t.numel() > 0 and t.stride(-1) != 1 and t.shape[-1] != 1:
        raise OsdnError(OSDN_ERR_INVALID_ARG, "the last dimension of a token tensor must be contiguous")
    return t.data_ptr()


def _handle(stream):
    """Handle of `stream`, or of the current device's current stream."""
    return _current_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def osdn_recur_fwd(params, x, gate, h0, lengths, h, final_h, checkpoints, stream=None):
    """Raw C-ABI call of the gated linear recurrence (every tensor preallocated; strides in params)."""
    _check(lib().osdn_recur_fwd(params, _ptr_rows(x), _ptr_rows(gate), _ptr(h0), _ptr(lengths), _ptr_rows(h),
                                _ptr(final_h), _ptr(checkpoints), _handle(stream)))


def osdn_recur_bwd_workspace_size(params: osdn_recur_params) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().osdn_recur_bwd_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def osdn_recur_bwd(params, x, gate, h0, lengths, dh, dfinal_h, checkpoints, dx, dgate, dh0, workspace, stream=None):
    """Raw C-ABI call of the recurrence's backward."""
    _check(lib().osdn_recur_bwd(params, _ptr_rows(x), _ptr_rows(gate), _ptr(h0), _ptr(lengths), _ptr_rows(dh),
                                _ptr(dfinal_h), _ptr(checkpoints), _ptr(dx), _ptr(dgate), _ptr(dh0), _ptr(workspace),
                                _ws_bytes(workspace), _handle(stream)))


def osdn_recur_step(params, x, gate, state, h, stream=None):
    """Raw C-ABI call: one token of the recurrence, state updated in place."""
    _check(lib().osdn_recur_step(params, _ptr_rows(x), _ptr_rows(gate), _ptr(state), _ptr_rows(h), _handle(stream)))


def osdn_qk_fwd(params, q, k, wq, wk, positions, freqs, lengths, q_out, k_out, stream=None):
    """Raw C-ABI call of the query and key norms with the rotation (strides in params)."""
    _check(lib().osdn_qk_fwd(params, _ptr_rows(q), _ptr_rows(k), _ptr(wq), _ptr(wk), _ptr(positions), _ptr(freqs),
                             _ptr(lengths), _ptr_rows(q_out), _ptr_rows(k_out), _handle(stream)))


def osdn_qk_bwd_workspace_size(params: osdn_qk_params) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().osdn_qk_bwd_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def osdn_qk_bwd(params, q, k, wq, wk, positions, freqs, lengths, dq_out, dk_out, dq, dk, dwq, dwk, workspace,
                stream=None):
    """Raw C-ABI call of the backward of osdn_qk_fwd."""
    _check(lib().osdn_qk_bwd(params, _ptr_rows(q), _ptr_rows(k), _ptr(wq), _ptr(wk), _ptr(positions), _ptr(freqs),
                             _ptr(lengths), _ptr_rows(dq_out), _ptr_rows(dk_out), _ptr(dq), _ptr(dk), _ptr(dwq),
                             _ptr(dwk), _ptr(workspace), _ws_bytes(workspace), _handle(stream)))


def osdn_rope(params, x, positions, freqs, lengths, out, inverse=False, stream=None):
    """Raw C-ABI call of the rotation alone."""
    _check(lib().osdn_rope(params, _ptr_rows(x), _ptr(positions), _ptr(freqs), _ptr(lengths), _ptr_rows(out),
                           1 if inverse else 0, _handle(stream)))


def osdn_rope_freqs(rot_dim, base, scaling, factor, original_length, low_turns, high_turns):
    """The rotation's frequencies (a list of rot_dim / 2 floats, computed on the host) and the amplitude."""
    if rot_dim < 2 or rot_dim > 256:
        raise OsdnError(OSDN_ERR_INVALID_ARG, "rot_dim must be even, 2 .. 256 (got %d)" % rot_dim)
    out, amplitude = (ctypes.c_double * (rot_dim // 2))(), ctypes.c_double(0.0)
    _check(lib().osdn_rope_freqs(rot_dim, base, scaling, factor, original_length, low_turns, high_turns, out,
                                 ctypes.byref(amplitude)))
    return list(out), amplitude.value


def osdn_sync_status(stream=None) -> int:
    return lib().osdn_sync_status(_stream(stream))


def osdn_set_wait_limit_ns(ns: int) -> None:
    """Upper bound on any device-side wait of kernels launched afterwards (0 = the 4 s default)."""
    lib().osdn_set_wait_limit_ns(int(ns))
