"""Thin Python binding of libla.so (argument marshalling only).

``fwd`` and ``bwd`` follow the signatures of the linear_attn page
(module neuralops.core.triton_kernels.linear_attn): ``fwd(q, k, v, is_causal=False,
phi="elu+1", eps=1e-6, cos_weight=None, sin_weight=None)`` and ``bwd(q, k, v, grad_out,
...) -> (dq, dk, dv)``.  The key/value head count is read from ``k.shape[1]``; when it is
smaller than ``q.shape[1]`` the call is grouped-query attention (module
neuralops.core.triton_kernels.gqa) with the expansion fused into the kernels, and dk, dv
come back with the key/value shape, summed over each group.  Inputs may be strided views
(last dimension contiguous, e.g. slices of a fused qkv projection): their strides go to
``la_fwd_strided`` / ``la_bwd_strided``; outputs are contiguous.

PyTorch supplies device memory and the current stream; every arithmetic step runs in
the library's CUDA kernels.  There is no fallback: if libla.so is missing or a call
fails, an exception says why.

``stream=`` enqueues a call on another stream than torch's current one.  The caller orders
that stream after whatever makes the inputs and lets whatever uses the results wait for it;
memory is safe either way: see ``_memory_on`` and ``_keep``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libla.so")

LA_OK, LA_ERR_ARG, LA_ERR_UNSUPPORTED, LA_ERR_ALIGN, LA_ERR_CUDA, LA_ERR_TIMEOUT, LA_ERR_WORKSPACE = range(7)
LA_F32, LA_BF16 = 0, 1
LA_PATH_SIMT, LA_PATH_TCGEN05 = 0, 1
PHI = {"elu+1": 0, "relu": 1, "identity": 2}
_NOT_BUILT = {"softmax_free"}

_lib = None


class LaStrides(ctypes.Structure):
    """la_strides: element strides of a [B, H, N, D] input along B, H, N."""
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("n", ctypes.c_longlong)]


class LaQkArgs(ctypes.Structure):
    """la_qk_args: norm and rotation of la_qk_norm_rope_*."""
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("normalize", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("rot", ctypes.c_int), ("axes", ctypes.c_int), ("sections", ctypes.POINTER(ctypes.c_int)),
                ("positions", ctypes.c_void_p), ("pos_strides", ctypes.POINTER(ctypes.c_longlong)),
                ("inv_freq", ctypes.c_void_p)]


class LaSsmArgs(ctypes.Structure):
    """la_ssm_args: inputs of la_ssm_*."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "dt", "B", "C", "z", "A", "skip", "dt_bias", "initial_state", "lengths")] + \
        [(n + "_strides", ctypes.POINTER(LaStrides)) for n in ("x", "dt", "B", "C", "z")] + \
        [(n, ctypes.c_int) for n in ("batch", "N", "E", "S", "G", "dtype", "softplus")]


class LaSsmGrads(ctypes.Structure):
    """la_ssm_grads: outputs of la_ssm_bwd."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "ddt", "dB", "dC", "dz", "dA", "dskip", "ddt_bias",
                                               "grad_initial_state")]


class LinearAttentionError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(what)


def load(path: str | None = None) -> ctypes.CDLL:
    """Open libla.so (built by ``efficient_transformer_gb300.build.build()``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libla.so not found at {p}: build it with "
                           "`python -m efficient_transformer_gb300.build` (no fallback exists)")
    lib = ctypes.CDLL(p)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.la_workspace_size.argtypes = [i, i, i, i, i, i, i, i, i]
    lib.la_workspace_size.restype = sz
    lib.la_kernel_path.argtypes = [i, i, i, i, i, i, i, i, i]
    lib.la_kernel_path.restype = i
    lib.la_workspace_size_v.argtypes = [i, i, i, i, i, i, i, i, i, i]
    lib.la_workspace_size_v.restype = sz
    lib.la_kernel_path_v.argtypes = [i, i, i, i, i, i, i, i, i, i]
    lib.la_kernel_path_v.restype = i
    lib.la_fwd_v.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp, vp, vp, sz, vp]
    lib.la_fwd_v.restype = i
    lib.la_bwd_v.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp, vp, vp, sz, vp, sz, vp]
    lib.la_bwd_v.restype = i
    lib.la_fwd.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, vp, vp, sz, vp]
    lib.la_fwd.restype = i
    lib.la_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, vp, vp, sz, vp]
    lib.la_bwd.restype = i
    lib.la_bwd_from_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, vp, vp, sz, vp, sz,
                                    vp]
    lib.la_bwd_from_fwd.restype = i
    sp = ctypes.POINTER(LaStrides)
    lib.la_fwd_strided.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, vp, sp, sp, sp, vp, sz, vp]
    lib.la_fwd_strided.restype = i
    lib.la_bwd_strided.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, vp, sp, sp, sp, sp,
                                   vp, sz, vp, sz, vp]
    lib.la_bwd_strided.restype = i
    lib.la_get_status.argtypes = [vp]
    lib.la_get_status.restype = i
    lib.la_status_str.argtypes = [i]
    lib.la_status_str.restype = ctypes.c_char_p
    lib.la_last_cuda_error.argtypes = []
    lib.la_last_cuda_error.restype = ctypes.c_char_p
    lib.la_lowrank_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.la_lowrank_fwd.restype = i
    lib.la_lowrank_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.la_lowrank_workspace_size.restype = sz
    lib.la_lowrank_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, sz, vp]
    lib.la_lowrank_fwd_t.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.la_lowrank_fwd_t.restype = i
    lib.la_lowrank_bwd_t.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp, sz, vp]
    lib.la_lowrank_bwd_t.restype = i
    lib.la_lowrank_bwd.restype = i
    lib.la_decay_workspace_size.argtypes = [i] * 8
    lib.la_decay_workspace_size.restype = sz
    lib.la_decay_kernel_path.argtypes = [i] * 8
    lib.la_decay_kernel_path.restype = i
    lib.la_decay_fwd.argtypes = [vp] * 8 + [i] * 7 + [f, sp, sp, sp, vp, sz, vp]
    lib.la_decay_fwd.restype = i
    lib.la_decay_bwd.argtypes = [vp] * 11 + [i] * 7 + [f, sp, sp, sp, sp, vp, sz, vp]
    lib.la_decay_bwd.restype = i
    lib.la_decay_step.argtypes = [vp] * 8 + [i] * 7 + [f, sp, sp, sp, vp]
    lib.la_decay_step.restype = i
    qp = ctypes.POINTER(LaQkArgs)
    lib.la_qk_norm_rope_fwd.argtypes = [vp] * 4 + [i] * 6 + [sp, sp, qp, vp]
    lib.la_qk_norm_rope_fwd.restype = i
    lib.la_qk_norm_rope_workspace_size.argtypes = [i] * 6
    lib.la_qk_norm_rope_workspace_size.restype = sz
    lib.la_qk_norm_rope_bwd.argtypes = [vp] * 8 + [i] * 6 + [sp, sp, sp, sp, qp, vp, sz, vp]
    lib.la_qk_norm_rope_bwd.restype = i
    lib.la_conv_fwd.argtypes = [vp] * 7 + [i] * 7 + [sp, vp]
    lib.la_conv_fwd.restype = i
    lib.la_conv_workspace_size.argtypes = [i] * 5
    lib.la_conv_workspace_size.restype = sz
    lib.la_conv_bwd.argtypes = [vp] * 11 + [i] * 7 + [sp, sp, vp, sz, vp]
    lib.la_conv_bwd.restype = i
    lib.la_conv_step.argtypes = [vp] * 7 + [i] * 7 + [sp, vp]
    lib.la_conv_step.restype = i
    ap, gp = ctypes.POINTER(LaSsmArgs), ctypes.POINTER(LaSsmGrads)
    lib.la_ssm_workspace_size.argtypes = [i] * 7
    lib.la_ssm_workspace_size.restype = sz
    lib.la_ssm_states_size.argtypes = [i] * 4
    lib.la_ssm_states_size.restype = sz
    lib.la_ssm_fwd.argtypes = [ap, vp, vp, vp, sz, vp, sz, vp]
    lib.la_ssm_fwd.restype = i
    lib.la_ssm_bwd.argtypes = [ap, vp, sp, vp, vp, sz, gp, vp, sz, vp]
    lib.la_ssm_bwd.restype = i
    lib.la_ssm_step.argtypes = [ap, vp, vp, vp, vp, i, vp]
    lib.la_ssm_step.restype = i
    lib.la_trace_start.argtypes = []
    lib.la_trace_start.restype = i
    lib.la_trace_stop.argtypes = []
    lib.la_trace_stop.restype = i
    lib.la_trace_collect.argtypes = []
    lib.la_trace_collect.restype = i
    lib.la_trace_kernel.argtypes = [i, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(i),
                                    ctypes.POINTER(ctypes.c_double)]
    lib.la_trace_kernel.restype = i
    if path is None:
        _lib = lib
    return lib


_SIZES = {"la_conv": "W must be 2, 3 or 4, E a multiple of 8", "la_ssm": "S must be 8, 16, 32 or 64, E / G a multiple of 8"}


def _raise(lib, status: int, call: str):
    what = lib.la_status_str(status).decode()
    if status == LA_ERR_UNSUPPORTED and call.rsplit("_", 1)[0] in _SIZES:
        what = "unsupported sizes: " + _SIZES[call.rsplit("_", 1)[0]]
    if status == LA_ERR_CUDA:
        what += ": " + lib.la_last_cuda_error().decode()
    raise LinearAttentionError(status, f"{call}: {what}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _phi_code(phi: str) -> int:
    if phi in _NOT_BUILT:
        raise NotImplementedError(f"phi={phi!r} is not built (only 'elu+1', 'relu' and 'identity')")
    if phi not in PHI:
        raise ValueError(f"unknown phi {phi!r}")
    return PHI[phi]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_inputs(q, k, v, cos_weight, sin_weight, extra=()):
    for name, t in (("q", q), ("k", k), ("v", v)) + tuple(extra):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1) or min(t.stride()) < 0:
            raise ValueError(f"{name} must be a [B, H, N, D] tensor whose last dimension is contiguous")
        if t.dtype != q.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, q has {q.dtype}")
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    B, Hq, N, D = q.shape
    if k.shape[0] != B or k.shape[2:] != (N, D) or v.shape[:3] != k.shape[:3]:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if (cos_weight is None) != (sin_weight is None):
        raise ValueError("give both cos_weight and sin_weight or neither")
    for name, w in (("cos_weight", cos_weight), ("sin_weight", sin_weight)):
        if w is not None and (w.dtype != torch.float32 or w.device != q.device or w.shape != (N,)
                              or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 CUDA vector of length N={N} on q's device")
    return B, Hq, k.shape[1], N, D, v.shape[3]


def _strides(t):
    """la_strides of an input (None when contiguous: the plain entry points take it)."""
    if t.is_contiguous():
        return None
    return ctypes.pointer(LaStrides(t.stride(0), t.stride(1), t.stride(2)))


def _stream_handle(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check_device(like, stream):
    """The raw stream of a call.  The library launches on the current device; the call's tensors, which lie on ``like``'s,
    and its stream must be of that one."""
    at, here = like.get_device(), torch.cuda.current_device()
    if at != here:
        raise ValueError(f"the tensors are on cuda:{at}, the current device is cuda:{here}: "
                         f"call under torch.cuda.device({at})")
    if stream is not None and stream.device.index != at:
        raise ValueError(f"the tensors are on cuda:{at}, the stream is one of {stream.device}")
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream().cuda_stream if _raw is None else _raw(here)


def workspace_size(B, Hq, Hkv, N, D, dtype: torch.dtype, is_causal: bool, has_weights: bool,
                   is_bwd: bool, Dv: int | None = None) -> int:
    code = LA_F32 if dtype == torch.float32 else LA_BF16
    return int(load().la_workspace_size_v(B, Hq, Hkv, N, D, D if Dv is None else Dv, code, int(is_causal),
                                          int(has_weights), int(is_bwd)))


def kernel_path(B, Hq, Hkv, N, D, dtype: torch.dtype, is_causal: bool, has_weights: bool,
                is_bwd: bool, Dv: int | None = None) -> int:
    code = LA_F32 if dtype == torch.float32 else LA_BF16
    return int(load().la_kernel_path_v(B, Hq, Hkv, N, D, D if Dv is None else Dv, code, int(is_causal),
                                       int(has_weights), int(is_bwd)))


_NO_SWITCH = contextlib.nullcontext()


def _memory_on(stream):
    """Context of a call's own allocations: memory of the stream that its kernels run on.  torch reuses a block in the
    order of the stream that it was allocated on, so scratch of the current stream could go to the next operation there
    while the kernels still use it, or come from an earlier one that has not finished."""
    return _NO_SWITCH if stream is None else torch.cuda.stream(stream)


def _keep(stream, out, given):
    """Tensors that a call on ``stream`` shares with the current stream (its outputs and what it was given): freed, their
    memory is not reused before both streams are done with it."""
    here = torch.cuda.current_stream()
    if here == stream:
        return
    for t in out:
        if t is not None:
            t.record_stream(here)
            t.record_stream(stream)
    for t in given:
        if t is not None:
            t.record_stream(stream)


def _workspace(nbytes: int, device, given):
    if nbytes == 0:
        return None
    if given is not None:
        if given.numel() * given.element_size() < nbytes:
            raise ValueError(f"workspace holds {given.numel() * given.element_size()} bytes, "
                             f"{nbytes} needed")
        if given.device != device or not given.is_contiguous():
            raise ValueError("workspace must be contiguous and on the inputs' device")
        return given
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, is_causal: bool = False,
        phi: str = "elu+1", eps: float = 1e-6, cos_weight: torch.Tensor | None = None,
        sin_weight: torch.Tensor | None = None, *, out: torch.Tensor | None = None,
        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Linear-attention forward; returns ``out`` [B, Hq, N, Dv] in the dtype of ``q`` (Dv =
    v's last dimension; with Dv != D the inputs must be contiguous)."""
    lib = load()
    B, Hq, Hkv, N, D, Dv = _check_inputs(q, k, v, cos_weight, sin_weight)
    _check_device(q, stream)
    oshape = (B, Hq, N, Dv)
    if out is not None and (tuple(out.shape) != oshape or out.dtype != q.dtype or out.device != q.device
                            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous {oshape} tensor of q's dtype on q's device")
    dt = _dtype_code(q)
    with _memory_on(stream):
        out = torch.empty(oshape, dtype=q.dtype, device=q.device) if out is None else out
        ws = _workspace(lib.la_workspace_size_v(B, Hq, Hkv, N, D, Dv, dt, int(is_causal),
                                                int(cos_weight is not None), 0), q.device, workspace)
    if stream is not None:
        _keep(stream, (out,), (q, k, v, cos_weight, sin_weight, workspace))
    nws = 0 if ws is None else ws.numel() * ws.element_size()
    strides = [_strides(t) for t in (q, k, v)]
    if Dv != D:
        if any(x is not None for x in strides):
            raise ValueError("with Dv != D, q, k and v must be contiguous")
        st = lib.la_fwd_v(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, Hq, Hkv, N, D, Dv, dt, int(is_causal),
                          _phi_code(phi), float(eps), _ptr(cos_weight), _ptr(sin_weight), _ptr(ws), nws,
                          _stream_handle(stream))
        call = "la_fwd_v"
    elif all(x is None for x in strides):
        st = lib.la_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, Hq, Hkv, N, D, dt, int(is_causal),
                        _phi_code(phi), float(eps), _ptr(cos_weight), _ptr(sin_weight), _ptr(ws), nws,
                        _stream_handle(stream))
        call = "la_fwd"
    else:
        st = lib.la_fwd_strided(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, Hq, Hkv, N, D, dt, int(is_causal),
                                _phi_code(phi), float(eps), _ptr(cos_weight), _ptr(sin_weight), *strides,
                                _ptr(ws), nws, _stream_handle(stream))
        call = "la_fwd_strided"
    if st != LA_OK:
        _raise(lib, st, call)
    return out


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, grad_out: torch.Tensor,
        is_causal: bool = False, phi: str = "elu+1", eps: float = 1e-6,
        cos_weight: torch.Tensor | None = None, sin_weight: torch.Tensor | None = None, *,
        dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
        dv: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
        fwd_workspace: torch.Tensor | None = None):
    """Linear-attention backward; returns ``(dq, dk, dv)`` with the shapes of q, k and v.

    ``fwd_workspace``: the workspace of the ``fwd`` call just made on the same inputs (ordered
    before this call); its per-segment states are then reused instead of recomputed
    (``la_bwd_from_fwd``).  The results are the same either way."""
    lib = load()
    B, Hq, Hkv, N, D, Dv = _check_inputs(q, k, v, cos_weight, sin_weight, (("grad_out", grad_out),))
    _check_device(q, stream)
    if tuple(grad_out.shape) != (B, Hq, N, Dv):
        raise ValueError("grad_out must have the shape of out ([B, Hq, N, Dv])")
    with _memory_on(stream):
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device) if dq is None else dq
        dk = torch.empty(k.shape, dtype=k.dtype, device=k.device) if dk is None else dk
        dv = torch.empty(v.shape, dtype=v.dtype, device=v.device) if dv is None else dv
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor like its input")
    dt = _dtype_code(q)
    with _memory_on(stream):
        ws = _workspace(lib.la_workspace_size_v(B, Hq, Hkv, N, D, Dv, dt, int(is_causal),
                                                int(cos_weight is not None), 1), q.device, workspace)
    nws = 0 if ws is None else ws.numel() * ws.element_size()
    if fwd_workspace is not None and fwd_workspace.device != q.device:
        raise ValueError("fwd_workspace must be on q's device")
    if stream is not None:
        _keep(stream, (dq, dk, dv), (q, k, v, grad_out, cos_weight, sin_weight, workspace, fwd_workspace))
    strides = [_strides(t) for t in (q, k, v, grad_out)]
    if Dv != D:
        if any(x is not None for x in strides):
            raise ValueError("with Dv != D, q, k, v and grad_out must be contiguous")
        fws = 0 if fwd_workspace is None else fwd_workspace.numel() * fwd_workspace.element_size()
        st = lib.la_bwd_v(_ptr(q), _ptr(k), _ptr(v), _ptr(grad_out), _ptr(dq), _ptr(dk), _ptr(dv),
                          B, Hq, Hkv, N, D, Dv, dt, int(is_causal), _phi_code(phi), float(eps),
                          _ptr(cos_weight), _ptr(sin_weight), _ptr(fwd_workspace), fws,
                          _ptr(ws), nws, _stream_handle(stream))
        call = "la_bwd_v"
    elif any(x is not None for x in strides):
        fws = 0 if fwd_workspace is None else fwd_workspace.numel() * fwd_workspace.element_size()
        st = lib.la_bwd_strided(_ptr(q), _ptr(k), _ptr(v), _ptr(grad_out), _ptr(dq), _ptr(dk), _ptr(dv),
                                B, Hq, Hkv, N, D, dt, int(is_causal), _phi_code(phi), float(eps),
                                _ptr(cos_weight), _ptr(sin_weight), *strides, _ptr(fwd_workspace), fws,
                                _ptr(ws), nws, _stream_handle(stream))
        call = "la_bwd_strided"
    elif fwd_workspace is None:
        st = lib.la_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(grad_out), _ptr(dq), _ptr(dk), _ptr(dv),
                        B, Hq, Hkv, N, D, dt, int(is_causal), _phi_code(phi), float(eps),
                        _ptr(cos_weight), _ptr(sin_weight), _ptr(ws), nws, _stream_handle(stream))
        call = "la_bwd"
    else:
        st = lib.la_bwd_from_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(grad_out), _ptr(dq), _ptr(dk), _ptr(dv),
                                 B, Hq, Hkv, N, D, dt, int(is_causal), _phi_code(phi), float(eps),
                                 _ptr(cos_weight), _ptr(sin_weight), _ptr(fwd_workspace),
                                 fwd_workspace.numel() * fwd_workspace.element_size(), _ptr(ws), nws,
                                 _stream_handle(stream))
        call = "la_bwd_from_fwd"
    if st != LA_OK:
        _raise(lib, st, call)
    return dq, dk, dv


def _check_lowrank(x, U, V, bias):
    for name, t in (("x", x), ("U", U), ("V", V)) + ((("bias", bias),) if bias is not None else ()):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if t.dtype != x.dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, x has {x.dtype}")
        if t.device != x.device:
            raise ValueError(f"{name} is on {t.device}, x on {x.device}")
    if U.dim() != 2 or V.dim() != 2 or x.shape[-1] != V.shape[1] or U.shape[1] != V.shape[0]:
        raise ValueError(f"shapes disagree: x {tuple(x.shape)}, U {tuple(U.shape)}, V {tuple(V.shape)}")
    if bias is not None and bias.shape != (U.shape[0],):
        raise ValueError("bias must have K_out = U.shape[0] elements")
    M = x.numel() // x.shape[-1]
    return M, V.shape[1], V.shape[0], U.shape[0]


def lowrank_fwd(x: torch.Tensor, U: torch.Tensor, V: torch.Tensor, bias: torch.Tensor | None = None, *,
                out: torch.Tensor | None = None, t_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Low-rank projection ``y = (x @ V.T) @ U.T + bias`` (module
    neuralops.core.triton_kernels.low_rank, ``fwd``): x [..., K_in], U [K_out, r], V [r, K_in];
    returns y [..., K_out].  ``t_out`` ([M, r], x's dtype): also receives the bottleneck
    t = x V^T for ``lowrank_bwd(..., t=t_out)`` (``la_lowrank_fwd_t``)."""
    lib = load()
    M, K_in, r, K_out = _check_lowrank(x, U, V, bias)
    _check_device(x, stream)
    if out is None:
        with _memory_on(stream):
            out = torch.empty(x.shape[:-1] + (K_out,), dtype=x.dtype, device=x.device)
    elif out.shape != x.shape[:-1] + (K_out,) or out.dtype != x.dtype or out.device != x.device \
            or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor [..., K_out] of x's dtype on x's device")
    if stream is not None:
        _keep(stream, (out, t_out), (x, U, V, bias))
    if t_out is None:
        st = lib.la_lowrank_fwd(_ptr(x), _ptr(U), _ptr(V), _ptr(bias), _ptr(out), M, K_in, r, K_out,
                                _dtype_code(x), _stream_handle(stream))
        call = "la_lowrank_fwd"
    else:
        if t_out.shape != (M, r) or t_out.dtype != x.dtype or not t_out.is_contiguous() or t_out.device != x.device:
            raise ValueError(f"t_out must be a contiguous CUDA tensor [{M}, {r}] of x's dtype on x's device")
        st = lib.la_lowrank_fwd_t(_ptr(x), _ptr(U), _ptr(V), _ptr(bias), _ptr(out), _ptr(t_out), M, K_in, r,
                                  K_out, _dtype_code(x), _stream_handle(stream))
        call = "la_lowrank_fwd_t"
    if st != LA_OK:
        _raise(lib, st, call)
    return out


def lowrank_bwd(x: torch.Tensor, U: torch.Tensor, V: torch.Tensor, grad_out: torch.Tensor,
                bias: torch.Tensor | None = None, *, workspace: torch.Tensor | None = None,
                t: torch.Tensor | None = None, stream=None):
    """Backward of ``lowrank_fwd`` (module neuralops.core.triton_kernels.low_rank, ``bwd``):
    returns ``(dx, dU, dV, dbias)``, dbias None without a bias.  ``t``: the bottleneck that
    ``lowrank_fwd(..., t_out=t)`` left for these x, V (``la_lowrank_bwd_t``: same results,
    one pass over x fewer)."""
    lib = load()
    M, K_in, r, K_out = _check_lowrank(x, U, V, bias)
    _check_device(x, stream)
    if grad_out.shape != x.shape[:-1] + (K_out,) or grad_out.dtype != x.dtype or grad_out.device != x.device \
            or not grad_out.is_contiguous():
        raise ValueError("grad_out must be a contiguous tensor [..., K_out] of x's dtype on x's device")
    dt = _dtype_code(x)
    with _memory_on(stream):
        dx, dU, dV = torch.empty_like(x), torch.empty_like(U), torch.empty_like(V)
        db = torch.empty_like(bias) if bias is not None else None
        ws = _workspace(lib.la_lowrank_workspace_size(M, K_in, r, K_out, dt, 1), x.device, workspace)
    if stream is not None:
        _keep(stream, (dx, dU, dV, db), (x, U, V, grad_out, bias, workspace, t))
    nws = 0 if ws is None else ws.numel() * ws.element_size()
    if t is None:
        st = lib.la_lowrank_bwd(_ptr(x), _ptr(U), _ptr(V), _ptr(grad_out), _ptr(dx), _ptr(dU), _ptr(dV), _ptr(db),
                                M, K_in, r, K_out, dt, _ptr(ws), nws, _stream_handle(stream))
        call = "la_lowrank_bwd"
    else:
        if t.shape != (M, r) or t.dtype != x.dtype or not t.is_contiguous() or t.device != x.device:
            raise ValueError(f"t must be a contiguous CUDA tensor [{M}, {r}] of x's dtype on x's device")
        st = lib.la_lowrank_bwd_t(_ptr(x), _ptr(U), _ptr(V), _ptr(t), _ptr(grad_out), _ptr(dx), _ptr(dU), _ptr(dV),
                                  _ptr(db), M, K_in, r, K_out, dt, _ptr(ws), nws, _stream_handle(stream))
        call = "la_lowrank_bwd_t"
    if st != LA_OK:
        _raise(lib, st, call)
    return dx, dU, dV, db


def decay_workspace_size(B, Hq, Hkv, N, D, dtype: torch.dtype, is_bwd: bool, Dv: int | None = None) -> int:
    code = LA_F32 if dtype == torch.float32 else LA_BF16
    return int(load().la_decay_workspace_size(B, Hq, Hkv, N, D, D if Dv is None else Dv, code, int(is_bwd)))


def decay_kernel_path(B, Hq, Hkv, N, D, dtype: torch.dtype, is_bwd: bool, Dv: int | None = None) -> int:
    code = LA_F32 if dtype == torch.float32 else LA_BF16
    return int(load().la_decay_kernel_path(B, Hq, Hkv, N, D, D if Dv is None else Dv, code, int(is_bwd)))


# The calls below can be as short as a few microseconds on the GPU, so their marshalling is kept small: addresses
# go as plain ints, sizes and strides that were asked for before come from caches (pure functions of their
# arguments), and the checks are one expression that names the culprit only when it fails.
def _addr(t):
    return None if t is None else t.data_ptr()


# torch's current stream as an integer, without a Stream object (2.8 of a call's 15 us) where torch has that
_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


@functools.lru_cache(maxsize=256)
def _strides_of(b, h, n):
    return ctypes.pointer(LaStrides(b, h, n))


def _stride_arg(t):
    return None if t.is_contiguous() else _strides_of(*t.stride()[:3])


@functools.lru_cache(maxsize=256)
def _decay_need(B, Hq, Hkv, N, D, Dv, dt, is_bwd):
    return int(load().la_decay_workspace_size(B, Hq, Hkv, N, D, Dv, dt, is_bwd))


@functools.lru_cache(maxsize=256)
def _qk_need(B, Hq, Hkv, N, D, dt):
    return int(load().la_qk_norm_rope_workspace_size(B, Hq, Hkv, N, D, dt))


def _rows_ok(t, dtype, device):
    """A [B, H, N, D] tensor of this dtype on CUDA device number `device`, D contiguous."""
    return t.dtype is dtype and t.get_device() == device >= 0 and t.dim() == 4 and (t.stride(3) == 1 or t.shape[3] == 1)


def _check_qkv(q, k, v, *extra):
    """(B, Hq, Hkv, N, D, Dv), as _check_inputs (which raises when something is wrong)."""
    try:
        dt, dev = q.dtype, q.get_device()
        if _rows_ok(q, dt, dev) and _rows_ok(k, dt, dev) and _rows_ok(v, dt, dev) and \
                (not extra or _rows_ok(extra[0], dt, dev)):
            B, Hq, N, D = q.shape
            _, Hkv, Nk, Dk = k.shape
            Dv = v.shape[3]
            if Nk == N and Dk == D and k.shape[0] == B and v.shape[:3] == k.shape[:3]:
                return B, Hq, Hkv, N, D, Dv
    except AttributeError:
        pass
    return _check_inputs(q, k, v, None, None, tuple(("grad_out", t) for t in extra))


def _check_vector(name, t, n, dtype, like):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != like.get_device() or t.dim() != 1 \
            or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} elements on q's device")


def _check_state(name, t, shape, like):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.get_device() != like.get_device() \
            or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor {shape} on q's device")


def _output(name, t, shape, like):
    if t is None:   # (empty_like is the quicker of the two by 1 to 2 us)
        return torch.empty_like(like) if like.shape == shape and like.is_contiguous() else like.new_empty(shape)
    if tuple(t.shape) != tuple(shape) or t.dtype != like.dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor of the inputs' dtype on their device")
    return t


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def decay_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *, scale: float = 1.0,
              initial_state: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
              lengths: torch.Tensor | None = None, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Linear attention with a decay for each key/value head, for prompts and training
    (``la_decay_fwd``): S_i = exp(log_decay) S_{i-1} + k_i v_i^T, out_i = scale q_i S_i.

    ``initial_state`` (float32 [B, Hkv, D, Dv]) is S before the first token, ``final_state``
    receives S after the last; they may be the same tensor.  ``lengths`` (int32 [B]): tokens of
    each sequence; out rows past them are zeros and what the inputs hold there is not used.
    Returns ``out`` [B, Hq, N, Dv].

    float32 inputs are computed in float32.  bfloat16 ones run on the tensor cores where D and Dv are 64
    or 128: sums and states in float32, each term of ``out`` rounded to bfloat16 once on its way; ``out`` is
    then 2.3e-3 from exact (2-norm; its own rounding alone 1.7e-3), ``final_state`` 3e-7."""
    lib = load()
    B, Hq, Hkv, N, D, Dv = _check_qkv(q, k, v)
    raw = _check_device(q, stream)
    dt = _dtype_code(q)
    _check_vector("log_decay", log_decay, Hkv, torch.float32, q)
    if lengths is not None:
        _check_vector("lengths", lengths, B, torch.int32, q)
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None:
            _check_state(name, t, (B, Hkv, D, Dv), q)
    with _memory_on(stream):
        out = _output("out", out, (B, Hq, N, Dv), q)
        ws = _workspace(_decay_need(B, Hq, Hkv, N, D, Dv, dt, 0), q.device, workspace)
    if stream is not None:
        _keep(stream, (out,), (q, k, v, log_decay, initial_state, final_state, lengths, workspace))
    st = lib.la_decay_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), log_decay.data_ptr(),
                          _addr(initial_state), _addr(final_state), _addr(lengths), B, Hq, Hkv, N, D, Dv, dt, scale,
                          _stride_arg(q), _stride_arg(k), _stride_arg(v), _addr(ws), _nbytes(ws), raw)
    if st != LA_OK:
        _raise(lib, st, "la_decay_fwd")
    return out


def decay_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, grad_out: torch.Tensor, log_decay: torch.Tensor, *,
              scale: float = 1.0, initial_state: torch.Tensor | None = None,
              grad_final_state: torch.Tensor | None = None, grad_initial_state: torch.Tensor | None = None,
              dq: torch.Tensor | None = None, dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None):
    """Gradient of ``decay_fwd`` (``la_decay_bwd``): returns ``(dq, dk, dv)``, dk and dv summed
    over each group's query heads.  ``grad_final_state`` is the gradient of the forward's
    final state (None: zeros); ``grad_initial_state``, when given, receives the initial state's.
    ``log_decay`` gets no gradient."""
    lib = load()
    B, Hq, Hkv, N, D, Dv = _check_qkv(q, k, v, grad_out)
    raw = _check_device(q, stream)
    if tuple(grad_out.shape) != (B, Hq, N, Dv):
        raise ValueError("grad_out must have the shape of out ([B, Hq, N, Dv])")
    dt = _dtype_code(q)
    _check_vector("log_decay", log_decay, Hkv, torch.float32, q)
    for name, t in (("initial_state", initial_state), ("grad_final_state", grad_final_state),
                    ("grad_initial_state", grad_initial_state)):
        if t is not None:
            _check_state(name, t, (B, Hkv, D, Dv), q)
    with _memory_on(stream):
        dq, dk, dv = _output("dq", dq, q.shape, q), _output("dk", dk, k.shape, k), _output("dv", dv, v.shape, v)
        ws = _workspace(_decay_need(B, Hq, Hkv, N, D, Dv, dt, 1), q.device, workspace)
    if stream is not None:
        _keep(stream, (dq, dk, dv), (q, k, v, grad_out, log_decay, initial_state, grad_final_state, grad_initial_state, workspace))
    st = lib.la_decay_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), grad_out.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                          dv.data_ptr(), log_decay.data_ptr(), _addr(initial_state), _addr(grad_final_state),
                          _addr(grad_initial_state), B, Hq, Hkv, N, D, Dv, dt, scale, _stride_arg(q), _stride_arg(k),
                          _stride_arg(v), _stride_arg(grad_out), _addr(ws), _nbytes(ws), raw)
    if st != LA_OK:
        _raise(lib, st, "la_decay_bwd")
    return dq, dk, dv


def decay_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, state: torch.Tensor, log_decay: torch.Tensor, *,
               slots: torch.Tensor | None = None, scale: float = 1.0, state_out: torch.Tensor | None = None,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One token of each sequence (``la_decay_step``): q [B, Hq, 1, D], k [B, Hkv, 1, D], v [B, Hkv,
    1, Dv] on a pool of states ``state`` (float32 [pool, Hkv, D, Dv]); sequence b owns slot
    ``slots[b]`` (int32 [B]; None: slot b), and a slot outside the pool marks a padding row (out
    zeros, no state touched).  The new states go to ``state_out`` at the same slots (None: into
    ``state``).  Returns ``out`` [B, Hq, 1, Dv]."""
    lib = load()
    B, Hq, Hkv, N, D, Dv = _check_qkv(q, k, v)
    raw = _check_device(q, stream)
    if N != 1:
        raise ValueError(f"decay_step takes one token per sequence (N = 1), got N = {N}")
    _check_vector("log_decay", log_decay, Hkv, torch.float32, q)
    if slots is not None:
        _check_vector("slots", slots, B, torch.int32, q)
    pool = state.shape[0] if state.dim() == 4 else 0
    _check_state("state", state, (pool, Hkv, D, Dv), q)
    if state_out is not None:
        _check_state("state_out", state_out, (pool, Hkv, D, Dv), q)
    with _memory_on(stream):
        out = _output("out", out, (B, Hq, 1, Dv), q)
    if stream is not None:
        _keep(stream, (out,), (q, k, v, state, log_decay, slots, state_out))
    st = lib.la_decay_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), state.data_ptr(),
                           (state if state_out is None else state_out).data_ptr(), log_decay.data_ptr(), _addr(slots),
                           pool, B, Hq, Hkv, D, Dv, _dtype_code(q), scale, _stride_arg(q), _stride_arg(k),
                           _stride_arg(v), raw)
    if st != LA_OK:
        _raise(lib, st, "la_decay_step")
    return out


def _check_qk(q, k, extra=()):
    try:
        dt, dev = q.dtype, q.get_device()
        if _rows_ok(q, dt, dev) and _rows_ok(k, dt, dev) and \
                (not extra or (_rows_ok(extra[0][1], dt, dev) and _rows_ok(extra[1][1], dt, dev))):
            B, Hq, N, D = q.shape
            Bk, Hkv, Nk, Dk = k.shape
            if Bk == B and Nk == N and Dk == D:
                return B, Hq, Hkv, N, D
    except AttributeError:
        pass
    for name, t in (("q", q), ("k", k)) + tuple(extra):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1) or min(t.stride()) < 0:
            raise ValueError(f"{name} must be a [B, H, N, D] tensor whose last dimension is contiguous")
        if t.dtype != q.dtype or t.device != q.device:
            raise TypeError(f"{name} must have q's dtype and device")
    B, Hq, N, D = q.shape
    if k.shape[0] != B or tuple(k.shape[2:]) != (N, D):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    return B, Hq, k.shape[1], N, D


@functools.lru_cache(maxsize=256)
def _sections_of(sections, pairs):
    """The host array of the axes' pairs; None where they do not add up."""
    return (ctypes.c_int * len(sections))(*sections) if sum(sections) == pairs else None


@functools.lru_cache(maxsize=256)
def _pos_strides_of(strides):
    return (ctypes.c_longlong * 3)(*strides)


def _qk_args(q, q_weight, k_weight, eps, positions, inv_freq, sections, interleaved, normalize):
    """la_qk_args of a call (and the host arrays that it points to)."""
    B, _, N, D = q.shape
    a = LaQkArgs(None, None, LA_F32, eps, normalize, interleaved)
    wt = None
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            t = w.dtype
            if (t is not torch.float32 and t is not q.dtype) or (wt is not None and t is not wt):
                raise TypeError(f"{name} must be float32 or of q's dtype, the same for both")
            wt = t
            _check_vector(name, w, D, t, q)
            setattr(a, name, w.data_ptr())
    if wt is torch.bfloat16:
        a.weight_dtype = LA_BF16
    if inv_freq is None:
        if positions is not None:
            raise ValueError("give both positions and inv_freq or neither")
        if sections is not None:
            raise ValueError("sections need positions and inv_freq")
        return a
    if positions is None:
        raise ValueError("give both positions and inv_freq or neither")
    pairs = inv_freq.numel()
    _check_vector("inv_freq", inv_freq, pairs, torch.float64, q)
    shape, strides = positions.shape, positions.stride()
    if len(shape) == 2:
        shape, strides = (1, *shape), (0, *strides)
    if positions.dtype is not torch.int64 or positions.get_device() != q.get_device() or len(shape) != 3 \
            or shape[1] != B or shape[2] != N:
        raise ValueError(f"positions must be an int64 tensor [axes, {B}, {N}] or [{B}, {N}] on q's device")
    axes = shape[0]
    if sections is None:
        if axes != 1:
            raise ValueError("several position axes need sections (pairs of each axis)")
        sections = (pairs,)
    host = _sections_of(tuple(sections), pairs) if len(sections) == axes else None
    if host is None:
        raise ValueError(f"sections {tuple(sections)} must name {axes} axes and add up to {pairs} pairs")
    a.rot, a.axes, a.sections = 2 * pairs, axes, host
    a.positions, a.inv_freq, a.pos_strides = positions.data_ptr(), inv_freq.data_ptr(), _pos_strides_of(strides)
    return a


def qk_norm_rope_fwd(q: torch.Tensor, k: torch.Tensor, *, q_weight: torch.Tensor | None = None,
                     k_weight: torch.Tensor | None = None, eps: float = 1e-6, positions: torch.Tensor | None = None,
                     inv_freq: torch.Tensor | None = None, sections=None, interleaved: bool = False,
                     normalize: bool = True, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     stream=None):
    """RMS norm of every head's query and key row, times its weight, then the rotation of
    positions, in one pass (``la_qk_norm_rope_fwd``); returns ``(q_out, k_out)``, contiguous.

    ``positions`` (int64 [B, N], or [axes, B, N] for up to four axes) times ``inv_freq`` (float64
    [rot / 2]) are the angles of the pairs; ``sections`` gives the pairs of each axis in turn.
    Pairs are (p, p + rot / 2), or (2p, 2p + 1) with ``interleaved``; elements past rot are not
    turned.  Without positions: the norm alone; with ``normalize=False``: the rotation alone."""
    lib = load()
    B, Hq, Hkv, N, D = _check_qk(q, k)
    raw = _check_device(q, stream)
    a = _qk_args(q, q_weight, k_weight, eps, positions, inv_freq, sections, interleaved, normalize)
    with _memory_on(stream):
        q_out, k_out = _output("q_out", q_out, q.shape, q), _output("k_out", k_out, k.shape, k)
    if stream is not None:
        _keep(stream, (q_out, k_out), (q, k, q_weight, k_weight, positions, inv_freq))
    st = lib.la_qk_norm_rope_fwd(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), B, Hq, Hkv, N, D,
                                 _dtype_code(q), _stride_arg(q), _stride_arg(k), ctypes.byref(a), raw)
    if st != LA_OK:
        _raise(lib, st, "la_qk_norm_rope_fwd")
    return q_out, k_out


def qk_norm_rope_workspace_size(B, Hq, Hkv, N, D, dtype: torch.dtype) -> int:
    code = LA_F32 if dtype == torch.float32 else LA_BF16
    return int(load().la_qk_norm_rope_workspace_size(B, Hq, Hkv, N, D, code))


def qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, grad_q: torch.Tensor, grad_k: torch.Tensor, *,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     positions: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None, sections=None,
                     interleaved: bool = False, normalize: bool = True, dq: torch.Tensor | None = None,
                     dk: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradient of ``qk_norm_rope_fwd`` for its inputs q, k and the gradients of its outputs
    (``la_qk_norm_rope_bwd``): returns ``(dq, dk, dq_weight, dk_weight)``, a weight's gradient None
    without that weight."""
    lib = load()
    B, Hq, Hkv, N, D = _check_qk(q, k, (("grad_q", grad_q), ("grad_k", grad_k)))
    raw = _check_device(q, stream)
    if grad_q.shape != q.shape or grad_k.shape != k.shape:
        raise ValueError("grad_q and grad_k must have the shapes of q and k")
    a = _qk_args(q, q_weight, k_weight, eps, positions, inv_freq, sections, interleaved, normalize)
    dt, ws = _dtype_code(q), None
    with _memory_on(stream):
        dq, dk = _output("dq", dq, q.shape, q), _output("dk", dk, k.shape, k)
        dqw = torch.empty_like(q_weight) if q_weight is not None else None
        dkw = torch.empty_like(k_weight) if k_weight is not None else None
        if dqw is not None or dkw is not None:
            ws = _workspace(_qk_need(B, Hq, Hkv, N, D, dt), q.device, workspace)
    if stream is not None:
        _keep(stream, (dq, dk, dqw, dkw), (q, k, grad_q, grad_k, q_weight, k_weight, positions, inv_freq, workspace))
    st = lib.la_qk_norm_rope_bwd(q.data_ptr(), k.data_ptr(), grad_q.data_ptr(), grad_k.data_ptr(), dq.data_ptr(),
                                 dk.data_ptr(), _addr(dqw), _addr(dkw), B, Hq, Hkv, N, D, dt, _stride_arg(q),
                                 _stride_arg(k), _stride_arg(grad_q), _stride_arg(grad_k), ctypes.byref(a), _addr(ws),
                                 _nbytes(ws), raw)
    if st != LA_OK:
        _raise(lib, st, "la_qk_norm_rope_bwd")
    return dq, dk, dqw, dkw


# ---- short causal convolution and selective state space scan -----------------------------------

def _check_tokens(name, t, shape, like):
    """A tensor [B, N, ..] of x's type on x's device, its last dimension contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != like.get_device() or t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor on x's device")
    if t.dtype is not like.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, x has {like.dtype}")
    if t.shape != shape or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a tensor {tuple(shape)} whose last dimension is contiguous, got {tuple(t.shape)}")


def _tokens_of(x):
    """(B, N, E) of x, checked."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a CUDA tensor [B, N, E]")
    _check_tokens("x", x, x.shape, x)
    return x.shape


def _token_strides(t):
    if t.is_contiguous():
        return None
    st = t.stride()
    return _strides_of(st[0], st[2] if len(st) == 4 else 0, st[1])


def _check_dense(name, t, shape, dtype, like):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != like.get_device() \
            or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)} on x's device")


_F32 = torch.float32


def _tokens_ok(t, shape, dtype, device):
    return t.dtype is dtype and t.get_device() == device and t.shape == shape and (t.is_contiguous() or t.stride(-1) == 1)


def _dense_ok(t, shape, dtype, device):
    return t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous()


def _conv_args(x, weight, bias):
    """(B, N, E, W, dtype code, weight's dtype code)"""
    try:   # (all at once; what is wrong is found out below)
        dev, ty, wty = x.get_device(), x.dtype, weight.dtype
        B, N, E = shape = x.shape
        Ew, W = weight.shape
        if dev >= 0 and Ew == E and (wty is ty or wty is _F32) and _tokens_ok(x, shape, ty, dev) and \
                _dense_ok(weight, weight.shape, wty, dev) and (bias is None or _dense_ok(bias, (E,), wty, dev)):
            return B, N, E, W, _dtype_code(x), LA_F32 if wty is _F32 else LA_BF16
    except (AttributeError, ValueError):
        pass
    B, N, E = _tokens_of(x)
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2 or weight.shape[0] != E or not weight.is_contiguous() \
            or weight.get_device() != x.get_device():
        raise ValueError(f"weight must be a contiguous tensor [{E}, W] on x's device")
    if weight.dtype is not torch.float32 and weight.dtype is not x.dtype:
        raise TypeError("weight must be float32 or of x's dtype")
    if bias is not None:
        _check_dense("bias", bias, (E,), weight.dtype, x)
    return B, N, E, weight.shape[1], _dtype_code(x), LA_F32 if weight.dtype is torch.float32 else LA_BF16


def conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *, silu: bool = True,
             initial_state: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
             lengths: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Short causal convolution of every channel (``la_conv_fwd``): x [B, N, E], weight [E, W] (W 2 to 4, float32 or x's
    dtype, bias [E] like it), out_t = silu(bias + sum_j weight[:, j] x_(t - W + 1 + j)), without the silu on request.

    ``initial_state`` ([B, W - 1, E], x's dtype) holds the rows before the first token, ``final_state`` receives the last
    W - 1; they may be the same tensor.  ``lengths`` (int32 [B]): tokens of each sequence; out rows past them are zeros and what
    x holds there is not used.  Returns ``out`` [B, N, E]."""
    lib = load()
    B, N, E, W, dt, wdt = _conv_args(x, weight, bias)
    raw = _check_device(x, stream)
    if lengths is not None:
        _check_dense("lengths", lengths, (B,), torch.int32, x)
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None:
            _check_dense(name, t, (B, W - 1, E), x.dtype, x)
    with _memory_on(stream):
        out = _output("out", out, (B, N, E), x)
    if stream is not None:
        _keep(stream, (out,), (x, weight, bias, initial_state, final_state, lengths))
    st = lib.la_conv_fwd(x.data_ptr(), weight.data_ptr(), _addr(bias), out.data_ptr(), _addr(initial_state),
                         _addr(final_state), _addr(lengths), B, N, E, W, dt, wdt, silu, _token_strides(x), raw)
    if st != LA_OK:
        _raise(lib, st, "la_conv_fwd")
    return out


@functools.lru_cache(maxsize=256)
def _conv_need(B, N, E, W, dt):
    return int(load().la_conv_workspace_size(B, N, E, W, dt))


def conv_workspace_size(B, N, E, W, dtype: torch.dtype) -> int:
    """Bytes of workspace of ``conv_bwd``."""
    return _conv_need(B, N, E, W, LA_F32 if dtype == torch.float32 else LA_BF16)


def conv_bwd(x: torch.Tensor, weight: torch.Tensor, grad_out: torch.Tensor, bias: torch.Tensor | None = None, *,
             silu: bool = True, initial_state: torch.Tensor | None = None, grad_final_state: torch.Tensor | None = None,
             grad_initial_state: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
             dx: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradient of ``conv_fwd`` (``la_conv_bwd``): returns ``(dx, dweight, dbias)``, dbias None without a bias.
    ``grad_final_state`` is the gradient of the final state (None: zeros); ``grad_initial_state``, when given, receives
    the initial state's (both of x's dtype)."""
    lib = load()
    B, N, E, W, dt, wdt = _conv_args(x, weight, bias)
    _check_tokens("grad_out", grad_out, x.shape, x)
    raw = _check_device(x, stream)
    if lengths is not None:
        _check_dense("lengths", lengths, (B,), torch.int32, x)
    for name, t in (("initial_state", initial_state), ("grad_final_state", grad_final_state),
                    ("grad_initial_state", grad_initial_state)):
        if t is not None:
            _check_dense(name, t, (B, W - 1, E), x.dtype, x)
    with _memory_on(stream):
        dx = _output("dx", dx, (B, N, E), x)
        dw = torch.empty_like(weight)
        db = torch.empty_like(bias) if bias is not None else None
        ws = _workspace(_conv_need(B, N, E, W, dt), x.device, workspace)
    if stream is not None:
        _keep(stream, (dx, dw, db), (x, weight, bias, grad_out, initial_state, grad_final_state, grad_initial_state, lengths,
                                     workspace))
    st = lib.la_conv_bwd(x.data_ptr(), weight.data_ptr(), _addr(bias), grad_out.data_ptr(), dx.data_ptr(), dw.data_ptr(),
                         _addr(db), _addr(initial_state), _addr(grad_final_state), _addr(grad_initial_state), _addr(lengths),
                         B, N, E, W, dt, wdt, silu, _token_strides(x), _token_strides(grad_out), _addr(ws), _nbytes(ws), raw)
    if st != LA_OK:
        _raise(lib, st, "la_conv_bwd")
    return dx, dw, db


def conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *,
              silu: bool = True, slots: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One token of each sequence through the convolution (``la_conv_step``): x [B, 1, E] on a pool of states ``state``
    ([pool, W - 1, E], x's dtype); slots, padding and ``state_out`` as in ``decay_step``.  Returns ``out`` [B, 1, E]."""
    lib = load()
    B, N, E, W, dt, wdt = _conv_args(x, weight, bias)
    raw = _check_device(x, stream)
    if N != 1:
        raise ValueError(f"conv_step takes one token per sequence (N = 1), got N = {N}")
    if slots is not None:
        _check_dense("slots", slots, (B,), torch.int32, x)
    pool = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 3 else 0
    _check_dense("state", state, (pool, W - 1, E), x.dtype, x)
    if state_out is not None:
        _check_dense("state_out", state_out, (pool, W - 1, E), x.dtype, x)
    with _memory_on(stream):
        out = _output("out", out, (B, 1, E), x)
    if stream is not None:
        _keep(stream, (out,), (x, state, weight, bias, slots, state_out))
    st = lib.la_conv_step(x.data_ptr(), weight.data_ptr(), _addr(bias), out.data_ptr(), state.data_ptr(),
                          (state if state_out is None else state_out).data_ptr(), _addr(slots), pool, B, E, W, dt, wdt, silu,
                          _token_strides(x), raw)
    if st != LA_OK:
        _raise(lib, st, "la_conv_step")
    return out


def _check_ssm(x, dt, A, B, C, skip, z, dt_bias, initial_state, lengths):
    """Raises for what is wrong with the inputs of a scan."""
    nB, N, E = _tokens_of(x)
    _check_tokens("dt", dt, x.shape, x)
    if not isinstance(B, torch.Tensor) or B.dim() != 4:
        raise ValueError("B must be a CUDA tensor [B, N, G, S]")
    G, S = B.shape[2:]
    _check_tokens("B", B, (nB, N, G, S), x)
    _check_tokens("C", C, (nB, N, G, S), x)
    _check_dense("A", A, (E, S), torch.float32, x)
    if z is not None:
        _check_tokens("z", z, x.shape, x)
    for name, t, shape, dtype in (("skip", skip, (E,), _F32), ("dt_bias", dt_bias, (E,), _F32),
                                  ("initial_state", initial_state, (nB, E, S), _F32), ("lengths", lengths, (nB,), torch.int32)):
        if t is not None:
            _check_dense(name, t, shape, dtype, x)


def _ssm_args(x, dt, A, B, C, skip, z, dt_bias, softplus, initial_state=None, lengths=None):
    """(la_ssm_args of a call, batch, N, E, S, G), checked."""
    try:   # (all at once; what is wrong is found out by _check_ssm)
        dev, ty = x.get_device(), x.dtype
        nB, N, E = shape = x.shape
        _, _, G, S = rows = B.shape
        if dev >= 0 and rows[0] == nB and rows[1] == N and _tokens_ok(x, shape, ty, dev) and _tokens_ok(dt, shape, ty, dev) and \
                _tokens_ok(B, rows, ty, dev) and _tokens_ok(C, rows, ty, dev) and _dense_ok(A, (E, S), _F32, dev) and \
                (z is None or _tokens_ok(z, shape, ty, dev)) and (skip is None or _dense_ok(skip, (E,), _F32, dev)) and \
                (dt_bias is None or _dense_ok(dt_bias, (E,), _F32, dev)) and \
                (initial_state is None or _dense_ok(initial_state, (nB, E, S), _F32, dev)) and \
                (lengths is None or _dense_ok(lengths, (nB,), torch.int32, dev)):
            return LaSsmArgs(x.data_ptr(), dt.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(z), A.data_ptr(), _addr(skip),
                             _addr(dt_bias), _addr(initial_state), _addr(lengths), _token_strides(x), _token_strides(dt),
                             _token_strides(B), _token_strides(C), None if z is None else _token_strides(z), nB, N, E, S, G,
                             _dtype_code(x), softplus), nB, N, E, S, G
    except (AttributeError, ValueError):
        pass
    _check_ssm(x, dt, A, B, C, skip, z, dt_bias, initial_state, lengths)
    raise ValueError("la_ssm: inputs do not fit together")


@functools.lru_cache(maxsize=256)
def _ssm_need(B, N, E, S, G, dt, is_bwd):
    return int(load().la_ssm_workspace_size(B, N, E, S, G, dt, is_bwd))


def ssm_workspace_size(B, N, E, S, G, dtype: torch.dtype, is_bwd: bool) -> int:
    """Bytes of workspace of ``ssm_fwd``, or of ``ssm_bwd`` (enough for both)."""
    return _ssm_need(B, N, E, S, G, LA_F32 if dtype == torch.float32 else LA_BF16, int(is_bwd))


@functools.lru_cache(maxsize=256)
def ssm_states_size(B, N, E, S) -> int:
    """Bytes of the states that ``ssm_fwd(..., states=)`` keeps for ``ssm_bwd``."""
    return int(load().la_ssm_states_size(B, N, E, S))


def _check_states(states, need, like):
    if not isinstance(states, torch.Tensor) or states.get_device() != like.get_device() or not states.is_contiguous() \
            or _nbytes(states) < need:
        raise ValueError(f"states must be a contiguous CUDA tensor of at least {need} bytes on x's device")


def ssm_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, *,
            skip: torch.Tensor | None = None, z: torch.Tensor | None = None, dt_bias: torch.Tensor | None = None,
            softplus: bool = True, initial_state: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
            lengths: torch.Tensor | None = None, states: torch.Tensor | None = None, out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Selective state space scan, for prompts and training (``la_ssm_fwd``): d_t = softplus(dt_t + dt_bias),
    h_t = exp(d_t A) h_(t-1) + d_t x_t B_t, out_t = (C_t . h_t + skip x_t) silu(z_t).

    x, dt, z [B, N, E] (z None: no gate); B, C [B, N, G, S], shared by the E / G channels of a group; A [E, S], skip and
    dt_bias [E] float32.  ``softplus=False``: d_t = dt_t + dt_bias.  ``initial_state`` (float32 [B, E, S]) is h before the first
    token, ``final_state`` receives h after the last; they may be the same tensor.  ``lengths`` (int32 [B]): tokens of each
    sequence; out rows past them are zeros and what the inputs hold there is not used.  ``states`` (at least
    ``ssm_states_size`` bytes) keeps what ``ssm_bwd`` needs.  Returns ``out`` [B, N, E].  Float32 arithmetic."""
    lib = load()
    a, nB, N, E, S, G = _ssm_args(x, dt, A, B, C, skip, z, dt_bias, softplus, initial_state, lengths)
    raw = _check_device(x, stream)
    if final_state is not None:
        _check_dense("final_state", final_state, (nB, E, S), torch.float32, x)
    if states is not None:
        _check_states(states, ssm_states_size(nB, N, E, S), x)
    with _memory_on(stream):
        out = _output("out", out, (nB, N, E), x)
        ws = _workspace(_ssm_need(nB, N, E, S, G, a.dtype, 0), x.device, workspace)
    if stream is not None:
        _keep(stream, (out,), (x, dt, A, B, C, skip, z, dt_bias, initial_state, final_state, lengths, states, workspace))
    st = lib.la_ssm_fwd(ctypes.byref(a), out.data_ptr(), _addr(final_state), _addr(states), _nbytes(states), _addr(ws),
                        _nbytes(ws), raw)
    if st != LA_OK:
        _raise(lib, st, "la_ssm_fwd")
    return out


def ssm_bwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, grad_out: torch.Tensor,
            *, skip: torch.Tensor | None = None, z: torch.Tensor | None = None, dt_bias: torch.Tensor | None = None,
            softplus: bool = True, initial_state: torch.Tensor | None = None,
            grad_final_state: torch.Tensor | None = None, grad_initial_state: torch.Tensor | None = None,
            lengths: torch.Tensor | None = None, states: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, stream=None):
    """Gradient of ``ssm_fwd`` (``la_ssm_bwd``): returns ``(dx, ddt, dA, dB, dC, dskip, dz, ddt_bias)``; dskip, dz and
    ddt_bias None without their inputs.  ``states``: those that ``ssm_fwd`` kept for these inputs (None: they are found
    again first, one more pass, from what ``initial_state`` holds now: not after a forward that replaced it).  ``grad_final_state`` is the gradient of the final state (None: zeros);
    ``grad_initial_state``, when given, receives the initial state's."""
    lib = load()
    a, nB, N, E, S, G = _ssm_args(x, dt, A, B, C, skip, z, dt_bias, softplus, initial_state, lengths)
    _check_tokens("grad_out", grad_out, x.shape, x)
    raw = _check_device(x, stream)
    if grad_final_state is not None:
        _check_dense("grad_final_state", grad_final_state, (nB, E, S), _F32, x)
    if grad_initial_state is not None:
        _check_dense("grad_initial_state", grad_initial_state, (nB, E, S), _F32, x)
    need, given = ssm_states_size(nB, N, E, S), states
    if states is not None:
        _check_states(states, need, x)
    with _memory_on(stream):   # (empty_like is the quickest)
        dx = torch.empty_like(x) if x.is_contiguous() else x.new_empty((nB, N, E))
        ddt = torch.empty_like(dx)
        dz = torch.empty_like(dx) if z is not None else None
        dB = torch.empty_like(B) if B.is_contiguous() else B.new_empty((nB, N, G, S))
        dC = torch.empty_like(dB)
        dA = torch.empty_like(A)
        dskip = torch.empty_like(skip) if skip is not None else None
        dbias = torch.empty_like(dt_bias) if dt_bias is not None else None
        ws = _workspace(_ssm_need(nB, N, E, S, G, a.dtype, 1), x.device, workspace)
        if states is None:
            states = torch.empty((need,), dtype=torch.uint8, device=x.device)
    if stream is not None:
        _keep(stream, (dx, ddt, dA, dB, dC, dskip, dz, dbias),
              (x, dt, A, B, C, grad_out, skip, z, dt_bias, initial_state, grad_final_state, grad_initial_state, lengths, given,
               workspace))
    if given is None:
        st = lib.la_ssm_fwd(ctypes.byref(a), None, None, states.data_ptr(), need, _addr(ws), _nbytes(ws), raw)
        if st != LA_OK:
            _raise(lib, st, "la_ssm_fwd")
    g = LaSsmGrads(dx.data_ptr(), ddt.data_ptr(), dB.data_ptr(), dC.data_ptr(), _addr(dz), dA.data_ptr(), _addr(dskip),
                   _addr(dbias), _addr(grad_initial_state))
    st = lib.la_ssm_bwd(ctypes.byref(a), grad_out.data_ptr(), _token_strides(grad_out), _addr(grad_final_state),
                        states.data_ptr(), _nbytes(states), ctypes.byref(g), _addr(ws), _nbytes(ws), raw)
    if st != LA_OK:
        _raise(lib, st, "la_ssm_bwd")
    return dx, ddt, dA, dB, dC, dskip, dz, dbias


def ssm_step(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, state: torch.Tensor, *,
             skip: torch.Tensor | None = None, z: torch.Tensor | None = None, dt_bias: torch.Tensor | None = None,
             softplus: bool = True, slots: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One token of each sequence through the scan (``la_ssm_step``): x, dt, z [B, 1, E], B, C [B, 1, G, S] on a pool of
    states ``state`` (float32 [pool, E, S]); slots, padding and ``state_out`` as in ``decay_step``.  Returns ``out`` [B, 1, E]."""
    lib = load()
    a, nB, N, E, S, G = _ssm_args(x, dt, A, B, C, skip, z, dt_bias, softplus)
    raw = _check_device(x, stream)
    if N != 1:
        raise ValueError(f"ssm_step takes one token per sequence (N = 1), got N = {N}")
    if slots is not None:
        _check_dense("slots", slots, (nB,), torch.int32, x)
    pool = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 3 else 0
    _check_dense("state", state, (pool, E, S), torch.float32, x)
    if state_out is not None:
        _check_dense("state_out", state_out, (pool, E, S), torch.float32, x)
    with _memory_on(stream):
        out = _output("out", out, (nB, 1, E), x)
    if stream is not None:
        _keep(stream, (out,), (x, dt, A, B, C, state, skip, z, dt_bias, slots, state_out))
    st = lib.la_ssm_step(ctypes.byref(a), out.data_ptr(), state.data_ptr(), (state if state_out is None else state_out).data_ptr(),
                         _addr(slots), pool, raw)
    if st != LA_OK:
        _raise(lib, st, "la_ssm_step")
    return out


def get_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel latched an error since the last check."""
    lib = load()
    st = lib.la_get_status(_stream_handle(stream))
    if st != LA_OK:
        _raise(lib, st, "la_get_status")


def trace_start() -> None:
    """Start bracketing every library kernel launch with CUDA events (for reports)."""
    load().la_trace_start()


def trace_stop() -> dict:
    """Stop tracing; return {kernel name: (launches, total device ms)} since trace_start()."""
    lib = load()
    lib.la_trace_stop()
    n = lib.la_trace_collect()
    res = {}
    for idx in range(n):
        name, launches, ms = ctypes.c_char_p(), ctypes.c_int(), ctypes.c_double()
        if lib.la_trace_kernel(idx, ctypes.byref(name), ctypes.byref(launches), ctypes.byref(ms)) == LA_OK:
            res[name.value.decode()] = (launches.value, ms.value)
    return res
