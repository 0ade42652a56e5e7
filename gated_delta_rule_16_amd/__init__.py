"""Python binding of libgdr, the gfx950 gated delta rule library.

Argument marshalling only: every step of every operation runs in the HIP
kernels behind the C ABI declared in ``include/gdr.h`` and (the operators
around the mixer) ``include/gdr_block.h``.  PyTorch supplies device memory
and the current HIP stream.  There is no CPU or PyTorch fallback — importing
this package without the built ``libgdr.so`` fails.

Functions mirror the C calls:

    gdr_chunk_fwd(q, k, v, alpha, beta, s0=None, ...)            -> (o, s_final)
    gdr_chunk_fwd_split(q, k, v, alpha, beta, s0=None, nseg=8, ...) -> (o, s_final)
    gdr_recurrent_step(q, k, v, alpha, beta, state, ...)         -> o
    gdr2_chunk_fwd(q, k, v, alpha, erase, write, s0=None, ...)   -> (o, s_final)
    gdr_output_gate(o, g, w=None, eps=1e-6, ...)                -> y
    gdr_output_gate_bwd(o, g, w, dy, eps=1e-6, ...)             -> (do, dg, dw)
    gdr_output_gate_bwd_noalloc(o, g, w, dy, eps=1e-6, ...)     -> (do, dg, dw)
    gdr_chunk_fwd_gate(q, k, v, alpha, beta, s0, g, w, eps, ...) -> (y, s_final)
    gdr_chunk_bwd(q, k, v, alpha, beta, s0, dout, ds_final=None)
        -> (dq, dk, dv, dalpha, dbeta, ds0)
    gdr2_chunk_bwd(q, k, v, alpha, erase, write, s0, dout, ds_final=None)
        -> (dq, dk, dv, dalpha, derase, dwrite, ds0)

    gdr_short_conv_fwd(x, w, bias=None, s0=None, ...)           -> (y, s_final)
    gdr_short_conv_step(x, w, bias, state, ...)                 -> y
    gdr_short_conv_bwd(x, w, bias, s0, dy, ds_final=None, ...)  -> (dx, dw, dbias, ds0)
    gdr_ssm_scan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, ...)
        -> (y, h_final)
    gdr_ssm_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, ...) -> y
    gdr_ssm_scan_bwd(x, dt, A, Bm, Cm, D, z, dt_bias, h0, dout, dh_final=None, ...)
        -> (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0)
    gdr_layer_norm_fwd(x, w=None, b=None, eps=1e-5, residual=None, ...) -> y or (y, h)
    gdr_layer_norm_bwd(x, w, dy, eps=1e-5, dres=None, ...)      -> (dx, dw, db)

``l2norm_qk=True`` calls the ``_ex`` variant of the same C function with
GDR_L2NORM_QK: q and k are L2-normalised on load inside the kernels.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch  # loads the HIP runtime libgdr.so binds to

__all__ = ["gdr_chunk_fwd", "gdr_recurrent_step", "gdr2_chunk_fwd", "gdr_output_gate",
           "gdr_chunk_bwd", "gdr_chunk_bwd_workspace_size",
           "gdr2_chunk_bwd", "gdr2_chunk_bwd_workspace_size",
           "gdr_chunk_fwd_split", "gdr_chunk_fwd_split_workspace_size",
           "gdr_output_gate_bwd", "gdr_output_gate_bwd_workspace_size",
           "gdr_output_gate_bwd_noalloc", "gdr_chunk_fwd_gate",
           "gdr_chunk_fwd_gate_workspace_size",
           "gdr_chunk_bwd_split", "gdr_chunk_bwd_split_workspace_size",
           "gdr2_chunk_fwd_split", "gdr2_chunk_bwd_split", "gdr2_chunk_bwd_split_workspace_size",
           "gdr_short_conv_fwd", "gdr_short_conv_step", "gdr_short_conv_bwd",
           "gdr_short_conv_bwd_workspace_size", "gdr_ssm_scan_fwd",
           "gdr_ssm_scan_fwd_workspace_size", "gdr_ssm_step", "gdr_ssm_scan_bwd",
           "gdr_ssm_scan_bwd_workspace_size", "gdr_layer_norm_fwd", "gdr_layer_norm_bwd",
           "gdr_layer_norm_bwd_workspace_size",
           "GdrError", "status_string", "lib", "LIB_PATH", "GDR_F32",
           "GDR_BF16", "GDR_L2NORM_QK", "GDR_SPLIT_FP32_STATES", "GDR_CONV_SILU",
           "GDR_SSM_SOFTPLUS", "GDR_SSM_MAX_N", "GDR_NORM_MAX_C"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "libgdr.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g;"
        f" g.build()'` (hipcc, gfx950) first")

lib = ctypes.CDLL(LIB_PATH)

GDR_F32, GDR_BF16 = 0, 1
GDR_L2NORM_QK = 1
GDR_SPLIT_FP32_STATES = 2
GDR_CONV_SILU = 1
GDR_SSM_SOFTPLUS = 1
GDR_SSM_MAX_N = 64
GDR_NORM_MAX_C = 1048576
_I64, _P, _E, _U = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32

lib.gdr_chunk_fwd.argtypes = [_I64] * 5 + [_E] + [_P] * 6 + [_E, _P, _P, _P]
lib.gdr_chunk_fwd.restype = ctypes.c_int
lib.gdr2_chunk_fwd.argtypes = [_I64] * 5 + [_E] + [_P] * 7 + [_E, _P, _P, _P]
lib.gdr2_chunk_fwd.restype = ctypes.c_int
lib.gdr_recurrent_step.argtypes = [_I64] * 4 + [_E] + [_P] * 6 + [_E, _P, _P]
lib.gdr_recurrent_step.restype = ctypes.c_int
lib.gdr_chunk_fwd_ex.argtypes = [_I64] * 5 + [_E] + [_P] * 6 + [_E, _P, _P, _U, _P]
lib.gdr_chunk_fwd_ex.restype = ctypes.c_int
lib.gdr2_chunk_fwd_ex.argtypes = [_I64] * 5 + [_E] + [_P] * 7 + [_E, _P, _P, _U, _P]
lib.gdr2_chunk_fwd_ex.restype = ctypes.c_int
lib.gdr_recurrent_step_ex.argtypes = [_I64] * 4 + [_E] + [_P] * 6 + [_E, _P, _U, _P]
lib.gdr_recurrent_step_ex.restype = ctypes.c_int
lib.gdr_output_gate.argtypes = [_I64] * 3 + [_E, _P, _E, _P, _P, ctypes.c_float, _E, _P, _P]
lib.gdr_output_gate.restype = ctypes.c_int
lib.gdr_chunk_bwd_workspace_size.argtypes = [_I64] * 5
lib.gdr_chunk_bwd_workspace_size.restype = ctypes.c_size_t
lib.gdr_chunk_bwd.argtypes = ([_I64] * 5 + [_E] + [_P] * 6 + [_E, _P, _P] + [_P] * 6 +
                              [_P, ctypes.c_size_t, _P])
lib.gdr_chunk_bwd.restype = ctypes.c_int
lib.gdr_chunk_bwd_ex.argtypes = ([_I64] * 5 + [_E] + [_P] * 6 + [_E, _P, _P] + [_P] * 6 +
                                 [_P, ctypes.c_size_t, _U, _P])
lib.gdr_chunk_bwd_ex.restype = ctypes.c_int
lib.gdr2_chunk_bwd_workspace_size.argtypes = [_I64] * 5
lib.gdr2_chunk_bwd_workspace_size.restype = ctypes.c_size_t
lib.gdr2_chunk_bwd.argtypes = ([_I64] * 5 + [_E] + [_P] * 7 + [_E, _P, _P] + [_P] * 7 +
                               [_P, ctypes.c_size_t, _P])
lib.gdr2_chunk_bwd.restype = ctypes.c_int
lib.gdr2_chunk_bwd_ex.argtypes = ([_I64] * 5 + [_E] + [_P] * 7 + [_E, _P, _P] + [_P] * 7 +
                                  [_P, ctypes.c_size_t, _U, _P])
lib.gdr2_chunk_bwd_ex.restype = ctypes.c_int
lib.gdr_chunk_fwd_split_workspace_size.argtypes = [_I64] * 5 + [_E, _I64]
lib.gdr_chunk_fwd_split_workspace_size.restype = ctypes.c_size_t
lib.gdr_chunk_fwd_split.argtypes = ([_I64] * 5 + [_E] + [_P] * 6 + [_E, _P, _P, _I64, _U, _P,
                                    ctypes.c_size_t, _P])
lib.gdr_chunk_fwd_split.restype = ctypes.c_int
lib.gdr_output_gate_bwd_workspace_size.argtypes = [_I64] * 3
lib.gdr_output_gate_bwd_workspace_size.restype = ctypes.c_size_t
lib.gdr_output_gate_bwd.argtypes = ([_I64] * 3 + [_E, _P, _E, _P, _P, ctypes.c_float, _E, _P] +
                                    [_P] * 4 + [ctypes.c_size_t, _P])
lib.gdr_output_gate_bwd.restype = ctypes.c_int
lib.gdr_output_gate_bwd_noalloc.argtypes = ([_I64] * 3 + [_E, _P, _E, _P, _P, ctypes.c_float, _E,
                                            _P] + [_P] * 3 + [_P])
lib.gdr_output_gate_bwd_noalloc.restype = ctypes.c_int
lib.gdr_chunk_fwd_gate_workspace_size.argtypes = [_I64] * 5 + [_E]
lib.gdr_chunk_fwd_gate_workspace_size.restype = ctypes.c_size_t
lib.gdr_chunk_fwd_gate.argtypes = ([_I64] * 5 + [_E] + [_P] * 6 + [_E, _P, _P, ctypes.c_float, _E,
                                   _P, _P, _U, _P, ctypes.c_size_t, _P])
lib.gdr_chunk_fwd_gate.restype = ctypes.c_int
lib.gdr_chunk_bwd_split_workspace_size.argtypes = [_I64] * 5 + [_E, _I64]
lib.gdr_chunk_bwd_split_workspace_size.restype = ctypes.c_size_t
lib.gdr_chunk_bwd_split.argtypes = ([_I64] * 5 + [_E] + [_P] * 6 + [_E, _P, _P] + [_P] * 6 +
                                    [_I64, _U, _P, ctypes.c_size_t, _P])
lib.gdr_chunk_bwd_split.restype = ctypes.c_int
lib.gdr2_chunk_fwd_split.argtypes = ([_I64] * 5 + [_E] + [_P] * 7 + [_E, _P, _P, _I64, _U, _P,
                                     ctypes.c_size_t, _P])
lib.gdr2_chunk_fwd_split.restype = ctypes.c_int
lib.gdr2_chunk_bwd_split_workspace_size.argtypes = [_I64] * 5 + [_E, _I64]
lib.gdr2_chunk_bwd_split_workspace_size.restype = ctypes.c_size_t
lib.gdr2_chunk_bwd_split.argtypes = ([_I64] * 5 + [_E] + [_P] * 7 + [_E, _P, _P] + [_P] * 7 +
                                     [_I64, _U, _P, ctypes.c_size_t, _P])
lib.gdr2_chunk_bwd_split.restype = ctypes.c_int
_F, _Z = ctypes.c_float, ctypes.c_size_t
lib.gdr_short_conv_fwd.argtypes = [_I64] * 4 + [_E] + [_P] * 5 + [_U, _E, _P, _P, _P]
lib.gdr_short_conv_fwd.restype = ctypes.c_int
lib.gdr_short_conv_step.argtypes = [_I64] * 3 + [_E, _P, _I64, _P, _P, _P, _U, _E, _P, _P]
lib.gdr_short_conv_step.restype = ctypes.c_int
lib.gdr_short_conv_bwd_workspace_size.argtypes = [_I64] * 4
lib.gdr_short_conv_bwd_workspace_size.restype = ctypes.c_size_t
lib.gdr_short_conv_bwd.argtypes = ([_I64] * 4 + [_E] + [_P] * 4 + [_E] + [_P] * 3 + [_U, _E] +
                                   [_P] * 5 + [_Z, _P])
lib.gdr_short_conv_bwd.restype = ctypes.c_int
lib.gdr_ssm_scan_fwd_workspace_size.argtypes = [_I64] * 5
lib.gdr_ssm_scan_fwd_workspace_size.restype = ctypes.c_size_t
lib.gdr_ssm_scan_fwd.argtypes = ([_I64] * 5 + [_E] + [_P] * 10 + [_U, _E] + [_P] * 3 + [_Z, _P])
lib.gdr_ssm_scan_fwd.restype = ctypes.c_int
lib.gdr_ssm_step.argtypes = [_I64] * 4 + [_E] + [_P] * 10 + [_U, _E, _P, _P]
lib.gdr_ssm_step.restype = ctypes.c_int
lib.gdr_ssm_scan_bwd_workspace_size.argtypes = [_I64] * 5
lib.gdr_ssm_scan_bwd_workspace_size.restype = ctypes.c_size_t
lib.gdr_ssm_scan_bwd.argtypes = ([_I64] * 5 + [_E] + [_P] * 9 + [_E] + [_P] * 3 + [_U, _E] +
                                 [_P] * 10 + [_Z, _P])
lib.gdr_ssm_scan_bwd.restype = ctypes.c_int
lib.gdr_layer_norm_fwd.argtypes = [_I64, _I64, _E, _P, _I64, _E, _P, _I64, _P, _P, _F, _E, _P, _P,
                                   _P]
lib.gdr_layer_norm_fwd.restype = ctypes.c_int
lib.gdr_layer_norm_bwd_workspace_size.argtypes = [_I64, _I64]
lib.gdr_layer_norm_bwd_workspace_size.restype = ctypes.c_size_t
lib.gdr_layer_norm_bwd.argtypes = [_I64, _I64, _E, _P, _I64, _P, _E, _P, _I64, _F, _E, _P, _I64,
                                   _P, _P, _P, _P, _Z, _P]
lib.gdr_layer_norm_bwd.restype = ctypes.c_int
lib.gdr_status_string.argtypes = [ctypes.c_int]
lib.gdr_status_string.restype = ctypes.c_char_p
lib.gdr_version.restype = ctypes.c_int

_DT = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16}


class GdrError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {status_string(code)} (status {code})")
        self.code = code


def status_string(code: int) -> str:
    return lib.gdr_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(name, t, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _run(name, code):
    if code != 0:
        raise GdrError(name, code)


def gdr_chunk_fwd(q, k, v, alpha, beta, s0=None, *, out_dtype=None, o=None,
                  s_final=None, want_state=True, l2norm_qk=False, stream=None):
    """Chunkwise gated delta rule forward.

    q, k [B,T,H,Dk]; v [B,T,H,Dv] (fp32 or bf16, same dtype); alpha, beta
    [B,T,H] fp32; s0 [B,H,Dv,Dk] fp32 or None.  ``out_dtype`` defaults to
    the input dtype.  Returns (o [B,T,H,Dv], s_final [B,H,Dv,Dk] or None).
    ``s_final`` may be passed in (it may be ``s0`` itself).
    """
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT:
        raise TypeError(f"unsupported input dtype {q.dtype}")
    _check("q", q, q.dtype, (B, T, H, Dk))
    _check("k", k, q.dtype, (B, T, H, Dk))
    _check("v", v, q.dtype, (B, T, H, Dv))
    _check("alpha", alpha, torch.float32, (B, T, H))
    _check("beta", beta, torch.float32, (B, T, H))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    odt = q.dtype if out_dtype is None else out_dtype
    if odt not in _DT:
        raise TypeError(f"unsupported output dtype {odt}")
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=odt, device=q.device)
    _check("o", o, odt, (B, T, H, Dv))
    if s_final is None and want_state:
        s_final = torch.empty((B, H, Dv, Dk), dtype=torch.float32, device=q.device)
    if s_final is not None:
        _check("s_final", s_final, torch.float32, (B, H, Dv, Dk))
    args = (B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v),
            _ptr(alpha), _ptr(beta), _ptr(s0), _DT[odt], _ptr(o), _ptr(s_final))
    if l2norm_qk:
        _run("gdr_chunk_fwd_ex", lib.gdr_chunk_fwd_ex(*args, GDR_L2NORM_QK, _stream(stream)))
    else:
        _run("gdr_chunk_fwd", lib.gdr_chunk_fwd(*args, _stream(stream)))
    return o, s_final


def gdr_chunk_fwd_gate_workspace_size(B, T, H, Dk, Dv, dtype) -> int:
    """Bytes of device workspace gdr_chunk_fwd_gate needs (0: none)."""
    return int(lib.gdr_chunk_fwd_gate_workspace_size(B, T, H, Dk, Dv, _DT[dtype]))


def gdr_chunk_fwd_gate(q, k, v, alpha, beta, s0, g, w=None, eps=1e-6, *, out_dtype=None, y=None,
                       s_final=None, want_state=True, l2norm_qk=False, workspace=None,
                       stream=None):
    """gdr_chunk_fwd followed by the output gate, y = o / sqrt(mean o^2 + eps)
    w SiLU(g), fused on the forward's stores (bf16 inputs).  g [B,T,H,Dv]
    fp32 or bf16, w [Dv] fp32 or None.  Returns (y [B,T,H,Dv], s_final or
    None); ``workspace`` (uint8 GPU tensor) is allocated here when None."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT or g.dtype not in _DT:
        raise TypeError("q and g must be float32 or bfloat16")
    _check("q", q, q.dtype, (B, T, H, Dk))
    _check("k", k, q.dtype, (B, T, H, Dk))
    _check("v", v, q.dtype, (B, T, H, Dv))
    _check("alpha", alpha, torch.float32, (B, T, H))
    _check("beta", beta, torch.float32, (B, T, H))
    _check("g", g, g.dtype, (B, T, H, Dv))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    if w is not None:
        _check("w", w, torch.float32, (Dv,))
    odt = q.dtype if out_dtype is None else out_dtype
    if odt not in _DT:
        raise TypeError(f"unsupported output dtype {odt}")
    if y is None:
        y = torch.empty((B, T, H, Dv), dtype=odt, device=q.device)
    _check("y", y, odt, (B, T, H, Dv))
    if s_final is None and want_state:
        s_final = torch.empty((B, H, Dv, Dk), dtype=torch.float32, device=q.device)
    if s_final is not None:
        _check("s_final", s_final, torch.float32, (B, H, Dv, Dk))
    if workspace is None:
        workspace = torch.empty(max(gdr_chunk_fwd_gate_workspace_size(B, T, H, Dk, Dv, q.dtype), 16),
                                dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8)
    _run("gdr_chunk_fwd_gate", lib.gdr_chunk_fwd_gate(
        B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
        _ptr(s0), _DT[g.dtype], _ptr(g), _ptr(w), float(eps), _DT[odt], _ptr(y), _ptr(s_final),
        GDR_L2NORM_QK if l2norm_qk else 0, _ptr(workspace), workspace.numel(), _stream(stream)))
    return y, s_final


def gdr_chunk_fwd_split_workspace_size(B, T, H, Dk, Dv, dtype, nseg) -> int:
    """Bytes of device workspace gdr_chunk_fwd_split needs (0: none)."""
    return int(lib.gdr_chunk_fwd_split_workspace_size(B, T, H, Dk, Dv, _DT[dtype], nseg))


def gdr_chunk_fwd_split(q, k, v, alpha, beta, s0=None, *, nseg=8, out_dtype=None, o=None,
                        s_final=None, want_state=True, l2norm_qk=False, workspace=None,
                        stream=None):
    """gdr_chunk_fwd with each sequence split into ``nseg`` segments that run
    side by side (T divisible by nseg).  Same arguments and results as
    gdr_chunk_fwd; ``workspace`` is a uint8 GPU tensor of at least
    gdr_chunk_fwd_split_workspace_size(...) bytes, allocated here when None."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT:
        raise TypeError(f"unsupported input dtype {q.dtype}")
    _check("q", q, q.dtype, (B, T, H, Dk))
    _check("k", k, q.dtype, (B, T, H, Dk))
    _check("v", v, q.dtype, (B, T, H, Dv))
    _check("alpha", alpha, torch.float32, (B, T, H))
    _check("beta", beta, torch.float32, (B, T, H))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    odt = q.dtype if out_dtype is None else out_dtype
    if odt not in _DT:
        raise TypeError(f"unsupported output dtype {odt}")
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=odt, device=q.device)
    _check("o", o, odt, (B, T, H, Dv))
    if s_final is None and want_state:
        s_final = torch.empty((B, H, Dv, Dk), dtype=torch.float32, device=q.device)
    if s_final is not None:
        _check("s_final", s_final, torch.float32, (B, H, Dv, Dk))
    need = gdr_chunk_fwd_split_workspace_size(B, T, H, Dk, Dv, q.dtype, nseg)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8)
    _run("gdr_chunk_fwd_split", lib.gdr_chunk_fwd_split(
        B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
        _ptr(s0), _DT[odt], _ptr(o), _ptr(s_final), nseg, GDR_L2NORM_QK if l2norm_qk else 0,
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return o, s_final


def gdr2_chunk_fwd(q, k, v, alpha, erase, write, s0=None, *, out_dtype=None,
                   o=None, s_final=None, want_state=True, l2norm_qk=False,
                   stream=None):
    """Chunkwise Gated Delta Rule-2 forward.

    q, k, alpha, erase [B,T,H,Dk]; v, write [B,T,H,Dv], all one dtype (fp32
    or bf16); s0 [B,H,Dv,Dk] fp32 or None.  Returns (o, s_final).
    """
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT:
        raise TypeError(f"unsupported input dtype {q.dtype}")
    for name, t, d in (("q", q, Dk), ("k", k, Dk), ("alpha", alpha, Dk),
                       ("erase", erase, Dk), ("v", v, Dv), ("write", write, Dv)):
        _check(name, t, q.dtype, (B, T, H, d))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    odt = q.dtype if out_dtype is None else out_dtype
    if odt not in _DT:
        raise TypeError(f"unsupported output dtype {odt}")
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=odt, device=q.device)
    _check("o", o, odt, (B, T, H, Dv))
    if s_final is None and want_state:
        s_final = torch.empty((B, H, Dv, Dk), dtype=torch.float32, device=q.device)
    if s_final is not None:
        _check("s_final", s_final, torch.float32, (B, H, Dv, Dk))
    args = (B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v),
            _ptr(alpha), _ptr(erase), _ptr(write), _ptr(s0), _DT[odt], _ptr(o),
            _ptr(s_final))
    if l2norm_qk:
        _run("gdr2_chunk_fwd_ex", lib.gdr2_chunk_fwd_ex(*args, GDR_L2NORM_QK, _stream(stream)))
    else:
        _run("gdr2_chunk_fwd", lib.gdr2_chunk_fwd(*args, _stream(stream)))
    return o, s_final


def gdr_recurrent_step(q, k, v, alpha, beta, state, *, out_dtype=None,
                       o=None, l2norm_qk=False, stream=None):
    """One decode token: q, k [N,H,Dk]; v [N,H,Dv]; alpha, beta [N,H] fp32;
    state [N,H,Dv,Dk] fp32, updated in place.  Returns o [N,H,Dv]."""
    N, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT:
        raise TypeError(f"unsupported input dtype {q.dtype}")
    _check("q", q, q.dtype, (N, H, Dk))
    _check("k", k, q.dtype, (N, H, Dk))
    _check("v", v, q.dtype, (N, H, Dv))
    _check("alpha", alpha, torch.float32, (N, H))
    _check("beta", beta, torch.float32, (N, H))
    _check("state", state, torch.float32, (N, H, Dv, Dk))
    odt = q.dtype if out_dtype is None else out_dtype
    if o is None:
        o = torch.empty((N, H, Dv), dtype=odt, device=q.device)
    _check("o", o, odt, (N, H, Dv))
    args = (N, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
            _ptr(beta), _ptr(state), _DT[odt], _ptr(o))
    if l2norm_qk:
        _run("gdr_recurrent_step_ex", lib.gdr_recurrent_step_ex(
            *args, GDR_L2NORM_QK, _stream(stream)))
    else:
        _run("gdr_recurrent_step", lib.gdr_recurrent_step(*args, _stream(stream)))
    return o


def gdr_output_gate(o, g, w=None, eps=1e-6, *, out_dtype=None, y=None, stream=None):
    """The block's output gate: y = o / sqrt(mean(o^2) + eps) * w * SiLU(g)
    over the last axis (Dv = 64 or 128).  o, g [..., H, Dv] (fp32 or bf16,
    each its own dtype); w [Dv] fp32 or None.  ``y`` may be ``o`` itself
    (same dtype) for an in-place gate.  Returns y."""
    if o.dim() < 2:
        raise ValueError("o must be [..., H, Dv]")
    H, Dv = o.shape[-2], o.shape[-1]
    N = o.numel() // (H * Dv) if H * Dv else 0
    for name, t in (("o", o), ("g", g)):
        if t.dtype not in _DT:
            raise TypeError(f"unsupported {name} dtype {t.dtype}")
    _check("o", o, o.dtype, tuple(o.shape))
    _check("g", g, g.dtype, tuple(o.shape))
    if w is not None:
        _check("w", w, torch.float32, (Dv,))
    if out_dtype is None:
        odt = o.dtype if y is None else y.dtype
    else:
        odt = out_dtype
    if odt not in _DT:
        raise TypeError(f"unsupported output dtype {odt}")
    if y is None:
        y = torch.empty(o.shape, dtype=odt, device=o.device)
    _check("y", y, odt, tuple(o.shape))
    _run("gdr_output_gate", lib.gdr_output_gate(
        N, H, Dv, _DT[o.dtype], _ptr(o), _DT[g.dtype], _ptr(g), _ptr(w), float(eps),
        _DT[odt], _ptr(y), _stream(stream)))
    return y


def gdr_chunk_bwd_workspace_size(B, T, H, Dk, Dv) -> int:
    """Bytes of device workspace gdr_chunk_bwd needs for these sizes."""
    return int(lib.gdr_chunk_bwd_workspace_size(B, T, H, Dk, Dv))


def gdr_chunk_bwd(q, k, v, alpha, beta, s0, dout, ds_final=None, *, workspace=None,
                  want_ds0=True, l2norm_qk=False, stream=None):
    """Reverse mode of gdr_chunk_fwd: returns fp32 (dq, dk, dv, dalpha,
    dbeta, ds0) for dL/do = ``dout`` [B,T,H,Dv] (fp32 or bf16) and
    dL/dS_T = ``ds_final`` [B,H,Dv,Dk] fp32 or None.  Inputs as for
    gdr_chunk_fwd.  ``workspace`` is a uint8 GPU tensor of at least
    gdr_chunk_bwd_workspace_size(...) bytes, allocated here when None.
    dq and dk are summed over blocks of state rows by atomic adds, so they
    can differ from run to run in the last bits."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT or dout.dtype not in _DT:
        raise TypeError("q and dout must be float32 or bfloat16")
    _check("q", q, q.dtype, (B, T, H, Dk))
    _check("k", k, q.dtype, (B, T, H, Dk))
    _check("v", v, q.dtype, (B, T, H, Dv))
    _check("alpha", alpha, torch.float32, (B, T, H))
    _check("beta", beta, torch.float32, (B, T, H))
    _check("dout", dout, dout.dtype, (B, T, H, Dv))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    if ds_final is not None:
        _check("ds_final", ds_final, torch.float32, (B, H, Dv, Dk))
    need = gdr_chunk_bwd_workspace_size(B, T, H, Dk, Dv)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty((B, T, H, Dk), **f32)
    dk = torch.empty((B, T, H, Dk), **f32)
    dv = torch.empty((B, T, H, Dv), **f32)
    da = torch.empty((B, T, H), **f32)
    db = torch.empty((B, T, H), **f32)
    ds0 = torch.empty((B, H, Dv, Dk), **f32) if want_ds0 else None
    args = (B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
            _ptr(s0), _DT[dout.dtype], _ptr(dout), _ptr(ds_final), _ptr(dq), _ptr(dk), _ptr(dv),
            _ptr(da), _ptr(db), _ptr(ds0), _ptr(workspace), workspace.numel())
    if l2norm_qk:
        _run("gdr_chunk_bwd_ex", lib.gdr_chunk_bwd_ex(*args, GDR_L2NORM_QK, _stream(stream)))
    else:
        _run("gdr_chunk_bwd", lib.gdr_chunk_bwd(*args, _stream(stream)))
    return dq, dk, dv, da, db, ds0


def gdr2_chunk_bwd_workspace_size(B, T, H, Dk, Dv) -> int:
    """Bytes of device workspace gdr2_chunk_bwd needs for these sizes."""
    return int(lib.gdr2_chunk_bwd_workspace_size(B, T, H, Dk, Dv))


def gdr2_chunk_bwd(q, k, v, alpha, erase, write, s0, dout, ds_final=None, *, workspace=None,
                   want_ds0=True, l2norm_qk=False, stream=None):
    """Reverse mode of gdr2_chunk_fwd: returns fp32 (dq, dk, dv, dalpha,
    derase, dwrite, ds0) for dL/do = ``dout`` [B,T,H,Dv] (fp32 or bf16) and
    dL/dS_T = ``ds_final`` [B,H,Dv,Dk] fp32 or None.  Inputs as for
    gdr2_chunk_fwd.  ``workspace`` is a uint8 GPU tensor of at least
    gdr2_chunk_bwd_workspace_size(...) bytes, allocated here when None."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT or dout.dtype not in _DT:
        raise TypeError("q and dout must be float32 or bfloat16")
    for name, x, d in (("q", q, Dk), ("k", k, Dk), ("v", v, Dv), ("alpha", alpha, Dk),
                       ("erase", erase, Dk), ("write", write, Dv)):
        _check(name, x, q.dtype, (B, T, H, d))
    _check("dout", dout, dout.dtype, (B, T, H, Dv))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    if ds_final is not None:
        _check("ds_final", ds_final, torch.float32, (B, H, Dv, Dk))
    need = gdr2_chunk_bwd_workspace_size(B, T, H, Dk, Dv)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty((B, T, H, Dk), **f32)
    dk = torch.empty((B, T, H, Dk), **f32)
    dv = torch.empty((B, T, H, Dv), **f32)
    da = torch.empty((B, T, H, Dk), **f32)
    de = torch.empty((B, T, H, Dk), **f32)
    dw = torch.empty((B, T, H, Dv), **f32)
    ds0 = torch.empty((B, H, Dv, Dk), **f32) if want_ds0 else None
    args = (B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(erase),
            _ptr(write), _ptr(s0), _DT[dout.dtype], _ptr(dout), _ptr(ds_final), _ptr(dq),
            _ptr(dk), _ptr(dv), _ptr(da), _ptr(de), _ptr(dw), _ptr(ds0), _ptr(workspace),
            workspace.numel())
    if l2norm_qk:
        _run("gdr2_chunk_bwd_ex", lib.gdr2_chunk_bwd_ex(*args, GDR_L2NORM_QK, _stream(stream)))
    else:
        _run("gdr2_chunk_bwd", lib.gdr2_chunk_bwd(*args, _stream(stream)))
    return dq, dk, dv, da, de, dw, ds0


def gdr_output_gate_bwd_workspace_size(N, H, Dv) -> int:
    """Bytes of device workspace gdr_output_gate_bwd needs for dw."""
    return int(lib.gdr_output_gate_bwd_workspace_size(N, H, Dv))


def gdr_output_gate_bwd(o, g, w, dy, eps=1e-6, *, want_dw=True, workspace=None, stream=None):
    """Reverse mode of gdr_output_gate: o, g, dy [..., H, Dv] (fp32 or bf16
    each), w [Dv] fp32 or None (ones).  Returns fp32 (do, dg, dw); dw [Dv]
    is None when ``want_dw`` is False."""
    if o.dim() < 2:
        raise ValueError("o must be [..., H, Dv]")
    H, Dv = o.shape[-2], o.shape[-1]
    N = o.numel() // (H * Dv) if o.numel() else 0
    for name, t in (("o", o), ("g", g), ("dy", dy)):
        if t.dtype not in _DT:
            raise TypeError(f"{name} must be float32 or bfloat16")
        _check(name, t, t.dtype, tuple(o.shape))
    if w is not None:
        _check("w", w, torch.float32, (Dv,))
    f32 = dict(dtype=torch.float32, device=o.device)
    do = torch.empty(o.shape, **f32)
    dg = torch.empty(o.shape, **f32)
    dw = torch.empty((Dv,), **f32) if want_dw else None
    if dw is not None and workspace is None:
        workspace = torch.empty(max(gdr_output_gate_bwd_workspace_size(N, H, Dv), 16),
                                dtype=torch.uint8, device=o.device)
    if workspace is not None:
        _check("workspace", workspace, torch.uint8)
    _run("gdr_output_gate_bwd", lib.gdr_output_gate_bwd(
        N, H, Dv, _DT[o.dtype], _ptr(o), _DT[g.dtype], _ptr(g), _ptr(w), float(eps),
        _DT[dy.dtype], _ptr(dy), _ptr(do), _ptr(dg), _ptr(dw), _ptr(workspace),
        0 if workspace is None else workspace.numel(), _stream(stream)))
    return do, dg, dw


def gdr_output_gate_bwd_noalloc(o, g, w, dy, eps=1e-6, *, want_dw=True, out=None, stream=None):
    """gdr_output_gate_bwd through the C call that takes no workspace (its
    dw partials go to the library's own per-GPU array).  ``out`` may give
    preallocated fp32 (do, dg, dw) tensors; otherwise they are created here.
    Returns (do, dg, dw), dw None when ``want_dw`` is False."""
    if o.dim() < 2:
        raise ValueError("o must be [..., H, Dv]")
    H, Dv = o.shape[-2], o.shape[-1]
    N = o.numel() // (H * Dv) if o.numel() else 0
    for name, t in (("o", o), ("g", g), ("dy", dy)):
        if t.dtype not in _DT:
            raise TypeError(f"{name} must be float32 or bfloat16")
        _check(name, t, t.dtype, tuple(o.shape))
    if w is not None:
        _check("w", w, torch.float32, (Dv,))
    if out is None:
        f32 = dict(dtype=torch.float32, device=o.device)
        out = (torch.empty(o.shape, **f32), torch.empty(o.shape, **f32),
               torch.empty((Dv,), **f32) if want_dw else None)
    do, dg, dw = out
    _check("do", do, torch.float32, tuple(o.shape))
    _check("dg", dg, torch.float32, tuple(o.shape))
    if dw is not None:
        _check("dw", dw, torch.float32, (Dv,))
    _run("gdr_output_gate_bwd_noalloc", lib.gdr_output_gate_bwd_noalloc(
        N, H, Dv, _DT[o.dtype], _ptr(o), _DT[g.dtype], _ptr(g), _ptr(w), float(eps),
        _DT[dy.dtype], _ptr(dy), _ptr(do), _ptr(dg), _ptr(dw), _stream(stream)))
    return do, dg, dw


def gdr_chunk_bwd_split_workspace_size(B, T, H, Dk, Dv, dtype, nseg) -> int:
    """Bytes of device workspace gdr_chunk_bwd_split needs."""
    return int(lib.gdr_chunk_bwd_split_workspace_size(B, T, H, Dk, Dv, _DT[dtype], nseg))


def gdr_chunk_bwd_split(q, k, v, alpha, beta, s0, dout, ds_final=None, *, nseg=8, workspace=None,
                        want_ds0=True, l2norm_qk=False, stream=None):
    """gdr_chunk_bwd with each sequence split into ``nseg`` segments that run
    side by side (T divisible by nseg).  Same arguments and results as
    gdr_chunk_bwd."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT or dout.dtype not in _DT:
        raise TypeError("q and dout must be float32 or bfloat16")
    _check("q", q, q.dtype, (B, T, H, Dk))
    _check("k", k, q.dtype, (B, T, H, Dk))
    _check("v", v, q.dtype, (B, T, H, Dv))
    _check("alpha", alpha, torch.float32, (B, T, H))
    _check("beta", beta, torch.float32, (B, T, H))
    _check("dout", dout, dout.dtype, (B, T, H, Dv))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    if ds_final is not None:
        _check("ds_final", ds_final, torch.float32, (B, H, Dv, Dk))
    need = gdr_chunk_bwd_split_workspace_size(B, T, H, Dk, Dv, q.dtype, nseg)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty((B, T, H, Dk), **f32)
    dk = torch.empty((B, T, H, Dk), **f32)
    dv = torch.empty((B, T, H, Dv), **f32)
    da = torch.empty((B, T, H), **f32)
    db = torch.empty((B, T, H), **f32)
    ds0 = torch.empty((B, H, Dv, Dk), **f32) if want_ds0 else None
    _run("gdr_chunk_bwd_split", lib.gdr_chunk_bwd_split(
        B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
        _ptr(s0), _DT[dout.dtype], _ptr(dout), _ptr(ds_final), _ptr(dq), _ptr(dk), _ptr(dv),
        _ptr(da), _ptr(db), _ptr(ds0), nseg, GDR_L2NORM_QK if l2norm_qk else 0,
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return dq, dk, dv, da, db, ds0


def gdr2_chunk_fwd_split(q, k, v, alpha, erase, write, s0=None, *, nseg=8, out_dtype=None,
                         o=None, s_final=None, want_state=True, l2norm_qk=False, workspace=None,
                         stream=None):
    """gdr2_chunk_fwd with each sequence split into ``nseg`` segments that
    run side by side (T divisible by nseg); workspace as for
    gdr_chunk_fwd_split."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT:
        raise TypeError(f"unsupported input dtype {q.dtype}")
    for name, x, d in (("q", q, Dk), ("k", k, Dk), ("v", v, Dv), ("alpha", alpha, Dk),
                       ("erase", erase, Dk), ("write", write, Dv)):
        _check(name, x, q.dtype, (B, T, H, d))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    odt = q.dtype if out_dtype is None else out_dtype
    if odt not in _DT:
        raise TypeError(f"unsupported output dtype {odt}")
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=odt, device=q.device)
    _check("o", o, odt, (B, T, H, Dv))
    if s_final is None and want_state:
        s_final = torch.empty((B, H, Dv, Dk), dtype=torch.float32, device=q.device)
    if s_final is not None:
        _check("s_final", s_final, torch.float32, (B, H, Dv, Dk))
    need = gdr_chunk_fwd_split_workspace_size(B, T, H, Dk, Dv, q.dtype, nseg)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8)
    _run("gdr2_chunk_fwd_split", lib.gdr2_chunk_fwd_split(
        B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(erase),
        _ptr(write), _ptr(s0), _DT[odt], _ptr(o), _ptr(s_final), nseg,
        GDR_L2NORM_QK if l2norm_qk else 0, _ptr(workspace), workspace.numel(), _stream(stream)))
    return o, s_final


def gdr2_chunk_bwd_split_workspace_size(B, T, H, Dk, Dv, dtype, nseg) -> int:
    """Bytes of device workspace gdr2_chunk_bwd_split needs."""
    return int(lib.gdr2_chunk_bwd_split_workspace_size(B, T, H, Dk, Dv, _DT[dtype], nseg))


def gdr2_chunk_bwd_split(q, k, v, alpha, erase, write, s0, dout, ds_final=None, *, nseg=8,
                         workspace=None, want_ds0=True, l2norm_qk=False, fp32_states=False,
                         stream=None):
    """gdr2_chunk_bwd with each sequence split into ``nseg`` segments that
    run side by side.  Same arguments and results as gdr2_chunk_bwd.
    ``fp32_states`` (GDR_SPLIT_FP32_STATES) runs the plain backward over
    the whole sequence instead (fp32 states throughout, no split)."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    if q.dtype not in _DT or dout.dtype not in _DT:
        raise TypeError("q and dout must be float32 or bfloat16")
    for name, x, d in (("q", q, Dk), ("k", k, Dk), ("v", v, Dv), ("alpha", alpha, Dk),
                       ("erase", erase, Dk), ("write", write, Dv)):
        _check(name, x, q.dtype, (B, T, H, d))
    _check("dout", dout, dout.dtype, (B, T, H, Dv))
    if s0 is not None:
        _check("s0", s0, torch.float32, (B, H, Dv, Dk))
    if ds_final is not None:
        _check("ds_final", ds_final, torch.float32, (B, H, Dv, Dk))
    need = gdr2_chunk_bwd_split_workspace_size(B, T, H, Dk, Dv, q.dtype, nseg)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("workspace", workspace, torch.uint8)
    f32 = dict(dtype=torch.float32, device=q.device)
    out = [torch.empty((B, T, H, d), **f32) for d in (Dk, Dk, Dv, Dk, Dk, Dv)]
    ds0 = torch.empty((B, H, Dv, Dk), **f32) if want_ds0 else None
    _run("gdr2_chunk_bwd_split", lib.gdr2_chunk_bwd_split(
        B, T, H, Dk, Dv, _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(erase),
        _ptr(write), _ptr(s0), _DT[dout.dtype], _ptr(dout), _ptr(ds_final),
        *[_ptr(x) for x in out], _ptr(ds0), nseg,
        (GDR_L2NORM_QK if l2norm_qk else 0) | (GDR_SPLIT_FP32_STATES if fp32_states else 0),
        _ptr(workspace), workspace.numel(), _stream(stream)))
    return tuple(out) + (ds0,)


# ---- operators around the mixer ------------------------------------------------
#
# Their inputs may be slices of wider tensors (any batch and token strides,
# channels contiguous), and they may live on another device than the current
# one: the call, and everything allocated for it, goes to the tensors' device
# and to ``stream`` (default: that device's current stream).


def _like(name, t, dtype, shape, device):
    """A tensor of this type and shape on ``device``."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.get_device() == device.index):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _row_strides(name, t, lead):
    """Element strides of the ``lead`` leading dimensions; the others must be
    contiguous."""
    st = t.stride()
    if len(st) == lead + 1:
        if st[-1] == 1:
            return st[:lead]
    elif st[-1] == 1 and st[-2] == t.shape[-1]:
        return st[:lead]
    shape = t.shape
    want = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] != 1 and st[i] != want and t.numel():
            raise ValueError(f"{name} must have contiguous channels")
        want *= shape[i]
    return st[:lead]


def _whole(name, t, dtype, shape, device):
    _like(name, t, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# a stream handle with no Stream object around it
_raw_stream = torch._C._cuda_getCurrentRawStream


def _on_own_device(fn):
    """Runs ``fn`` with its first tensor's device current, and with ``stream``
    (default: that device's current stream) as the current stream, so that
    what it allocates belongs there too."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        x = args[0] if args else kw.get("x")
        if isinstance(x, torch.Tensor) and x.is_cuda:
            if stream is not None:
                if stream.device != x.device:
                    raise ValueError(f"stream must be on {x.device}, got {stream.device}")
                with torch.cuda.stream(stream):
                    return fn(*args, **kw)
            if x.get_device() != torch._C._cuda_getDevice():
                with torch.cuda.device(x.device):
                    return fn(*args, **kw)
        return fn(*args, **kw)
    return call


def _first(name, t, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if t.dtype not in _DT:
        raise TypeError(f"unsupported {name} dtype {t.dtype}")
    return t.device


def _dt_of(name, dtype):
    if dtype not in _DT:
        raise TypeError(f"unsupported {name} {dtype}")
    return _DT[dtype]


def _buffer(name, t, dtype, shape, device, like=None):
    """A given output buffer, checked, or a new one (``like``: a tensor that may
    have its type and shape already, which is the quicker way to one)."""
    if t is None:
        return _new(like, dtype, shape, device)
    _whole(name, t, dtype, shape, device)
    return t


def _scratch(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    _like("workspace", workspace, torch.uint8, workspace.shape, device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _new(like, dtype, shape, device):
    """A new tensor; from ``like`` where that has its shape (half the host time)."""
    if like is not None and like.shape == shape and like.is_contiguous():
        return torch.empty_like(like, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=device)


@functools.lru_cache(maxsize=256)
def _need(name, *sizes):
    """A workspace size (a function of the sizes alone)."""
    return int(getattr(lib, name)(*sizes))


def _p(t):
    return None if t is None else t.data_ptr()


def _i64s(*v):
    return (ctypes.c_int64 * len(v))(*v)


@_on_own_device
def gdr_short_conv_fwd(x, w, bias=None, s0=None, *, silu=True, out_dtype=None, y=None,
                       s_final=None, want_state=True, stream=None):
    """Short causal depthwise convolution (with SiLU) over whole sequences.

    x [B,T,C] fp32 or bf16 (batch and token strides free); w [C,K] fp32, K = 2,
    3 or 4; bias [C] fp32 or None; s0 [B,K-1,C] in x's dtype or None: the inputs
    before x.  Returns (y [B,T,C], s_final [B,K-1,C] or None); ``s_final`` may
    be passed in (it may be ``s0`` itself)."""
    dev = _first("x", x, 3)
    B, T, C = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [C, K] tensor")
    K = w.shape[1]
    xs = _row_strides("x", x, 2)
    _whole("w", w, torch.float32, (C, K), dev)
    if bias is not None:
        _whole("bias", bias, torch.float32, (C,), dev)
    if s0 is not None:
        _whole("s0", s0, x.dtype, (B, K - 1, C), dev)
    odt = out_dtype or (x.dtype if y is None else y.dtype)
    code = _dt_of("output dtype", odt)
    y = _buffer("y", y, odt, (B, T, C), dev, x)
    if s_final is not None or want_state:
        s_final = _buffer("s_final", s_final, x.dtype, (B, max(K - 1, 0), C), dev, s0)
    _run("gdr_short_conv_fwd", lib.gdr_short_conv_fwd(
        B, T, C, K, _DT[x.dtype], _p(x), _i64s(*xs), _p(w), _p(bias), _p(s0),
        GDR_CONV_SILU if silu else 0, code, _p(y), _p(s_final), _raw_stream(dev.index)))
    return y, s_final


@_on_own_device
def gdr_short_conv_step(x, w, bias, state, *, silu=True, out_dtype=None, y=None, stream=None):
    """One decode token of gdr_short_conv_fwd: x [N,C], state [N,K-1,C] in x's
    dtype, moved on in place.  Returns y [N,C]."""
    dev = _first("x", x, 2)
    N, C = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [C, K] tensor")
    K = w.shape[1]
    xs = _row_strides("x", x, 1)
    _whole("w", w, torch.float32, (C, K), dev)
    if bias is not None:
        _whole("bias", bias, torch.float32, (C,), dev)
    _whole("state", state, x.dtype, (N, K - 1, C), dev)
    odt = out_dtype or (x.dtype if y is None else y.dtype)
    code = _dt_of("output dtype", odt)
    y = _buffer("y", y, odt, (N, C), dev, x)
    _run("gdr_short_conv_step", lib.gdr_short_conv_step(
        N, C, K, _DT[x.dtype], _p(x), xs[0], _p(w), _p(bias), _p(state),
        GDR_CONV_SILU if silu else 0, code, _p(y), _raw_stream(dev.index)))
    return y


def gdr_short_conv_bwd_workspace_size(B, T, C, K) -> int:
    """Bytes of device workspace gdr_short_conv_bwd needs for dw and dbias."""
    return int(lib.gdr_short_conv_bwd_workspace_size(B, T, C, K))


@_on_own_device
def gdr_short_conv_bwd(x, w, bias, s0, dy, ds_final=None, *, silu=True,
                       grad_dtype=torch.float32, want_dw=True, want_ds0=True, workspace=None,
                       stream=None):
    """Reverse mode of gdr_short_conv_fwd for dL/dy = ``dy`` [B,T,C] (fp32 or
    bf16, strides free) and dL/ds_final = ``ds_final`` [B,K-1,C] fp32 or None.
    Returns (dx [B,T,C] in ``grad_dtype``, dw [C,K], dbias [C], ds0 [B,K-1,C]),
    the last three fp32; dw and dbias are None without ``want_dw``, dbias also
    without bias, ds0 without ``want_ds0``."""
    dev = _first("x", x, 3)
    B, T, C = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [C, K] tensor")
    K = w.shape[1]
    xs = _row_strides("x", x, 2)
    _whole("w", w, torch.float32, (C, K), dev)
    if bias is not None:
        _whole("bias", bias, torch.float32, (C,), dev)
    if s0 is not None:
        _whole("s0", s0, x.dtype, (B, K - 1, C), dev)
    _first("dy", dy, 3)
    _like("dy", dy, dy.dtype, (B, T, C), dev)
    ys = _row_strides("dy", dy, 2)
    if ds_final is not None:
        _whole("ds_final", ds_final, torch.float32, (B, K - 1, C), dev)
    code = _dt_of("grad_dtype", grad_dtype)
    f32 = torch.float32
    dx = _new(dy, grad_dtype, x.shape, dev)
    dw = torch.empty_like(w) if want_dw else None
    db = torch.empty_like(bias) if want_dw and bias is not None else None
    ds0 = _new(ds_final, f32, (B, max(K - 1, 0), C), dev) if want_ds0 else None
    if want_dw or workspace is not None:
        workspace = _scratch(workspace, _need("gdr_short_conv_bwd_workspace_size", B, T, C, K),
                             dev)
    _run("gdr_short_conv_bwd", lib.gdr_short_conv_bwd(
        B, T, C, K, _DT[x.dtype], _p(x), _p(w), _p(bias), _p(s0), _DT[dy.dtype], _p(dy),
        _i64s(*xs, *ys), _p(ds_final), GDR_CONV_SILU if silu else 0, code, _p(dx), _p(dw),
        _p(db), _p(ds0), _p(workspace), 0 if workspace is None else workspace.numel(),
        _raw_stream(dev.index)))
    return dx, dw, db, ds0


def _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, lead):
    """Checks shared by the scan's calls; returns (device, sizes, strides)."""
    dev = _first("x", x, lead + 1)
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [D, N] tensor")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != lead + 2:
        raise ValueError("Bm must be [..., G, N]")
    Dn, N = A.shape
    G = Bm.shape[-2]
    dtype, shape = x.dtype, x.shape
    rows = shape[:lead]
    if shape[-1] != Dn:
        raise ValueError(f"x must have {Dn} channels, got {shape[-1]}")
    _like("dt", dt, dtype, shape, dev)
    _like("Bm", Bm, dtype, rows + (G, N), dev)
    _like("Cm", Cm, dtype, Bm.shape, dev)
    st = [*_row_strides("x", x, lead), *_row_strides("dt", dt, lead),
          *_row_strides("Bm", Bm, lead), *_row_strides("Cm", Cm, lead)]
    if z is None:
        st += [0] * lead
    else:
        _like("z", z, dtype, shape, dev)
        st += _row_strides("z", z, lead)
    _whole("A", A, torch.float32, (Dn, N), dev)
    if D is not None:
        _whole("D", D, torch.float32, (Dn,), dev)
    if dt_bias is not None:
        _whole("dt_bias", dt_bias, torch.float32, (Dn,), dev)
    return dev, (*rows, Dn, G, N), st


def gdr_ssm_scan_fwd_workspace_size(B, T, D, G, N) -> int:
    """Bytes of device workspace gdr_ssm_scan_fwd needs (0: none)."""
    return int(lib.gdr_ssm_scan_fwd_workspace_size(B, T, D, G, N))


@_on_own_device
def gdr_ssm_scan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, *, softplus=True,
                     out_dtype=None, y=None, h_final=None, want_state=True, workspace=None,
                     stream=None):
    """Selective state space scan over whole sequences: with Delta =
    softplus(dt + dt_bias), h_t = exp(Delta_t A) h_{t-1} + Delta_t x_t B_t,
    y_t = C_t . h_t + D x_t, times SiLU(z_t) when z is given.

    x, dt, z [B,T,D] and Bm, Cm [B,T,G,N], all one dtype (fp32 or bf16; batch
    and token strides free); A [D,N], D [D], dt_bias [D] fp32; h0 [B,D,N] fp32
    or None.  Returns (y [B,T,D], h_final [B,D,N] or None); ``h_final`` may be
    passed in (it may be ``h0`` itself)."""
    dev, (B, T, Dn, G, N), st = _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, 2)
    if h0 is not None:
        _whole("h0", h0, torch.float32, (B, Dn, N), dev)
    odt = out_dtype or (x.dtype if y is None else y.dtype)
    code = _dt_of("output dtype", odt)
    need = _need("gdr_ssm_scan_fwd_workspace_size", B, T, Dn, G, N)
    y = _buffer("y", y, odt, (B, T, Dn), dev, dt)
    if h_final is not None or want_state:
        h_final = _buffer("h_final", h_final, torch.float32, (B, Dn, N), dev, h0)
    if need or workspace is not None:
        workspace = _scratch(workspace, need, dev)
    _run("gdr_ssm_scan_fwd", lib.gdr_ssm_scan_fwd(
        B, T, Dn, G, N, _DT[x.dtype], _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D), _p(z),
        _p(dt_bias), _p(h0), _i64s(*st), GDR_SSM_SOFTPLUS if softplus else 0, code, _p(y),
        _p(h_final), _p(workspace), 0 if workspace is None else workspace.numel(),
        _raw_stream(dev.index)))
    return y, h_final


@_on_own_device
def gdr_ssm_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, *, softplus=True,
                 out_dtype=None, y=None, stream=None):
    """One decode token of gdr_ssm_scan_fwd: x, dt, z [N,D], Bm, Cm [N,G,S] for
    N sequences and S states; state [N,D,S] fp32, updated in place.  Returns
    y [N,D]."""
    dev, (Nq, Dn, G, N), st = _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, 1)
    _whole("state", state, torch.float32, (Nq, Dn, N), dev)
    odt = out_dtype or (x.dtype if y is None else y.dtype)
    code = _dt_of("output dtype", odt)
    y = _buffer("y", y, odt, (Nq, Dn), dev, dt)
    _run("gdr_ssm_step", lib.gdr_ssm_step(
        Nq, Dn, G, N, _DT[x.dtype], _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D), _p(z),
        _p(dt_bias), _p(state), _i64s(*st), GDR_SSM_SOFTPLUS if softplus else 0, code, _p(y),
        _raw_stream(dev.index)))
    return y


def gdr_ssm_scan_bwd_workspace_size(B, T, D, G, N) -> int:
    """Bytes of device workspace gdr_ssm_scan_bwd needs."""
    return int(lib.gdr_ssm_scan_bwd_workspace_size(B, T, D, G, N))


@_on_own_device
def gdr_ssm_scan_bwd(x, dt, A, Bm, Cm, D, z, dt_bias, h0, dout, dh_final=None, *, softplus=True,
                     grad_dtype=torch.float32, want_dh0=True, workspace=None, stream=None):
    """Reverse mode of gdr_ssm_scan_fwd for dL/dy = ``dout`` [B,T,D] (fp32 or
    bf16, strides free) and dL/dh_final = ``dh_final`` [B,D,N] fp32 or None.
    Returns (dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0): dx, ddt, dB, dC, dz
    in ``grad_dtype``, the others fp32; None for D, z, dt_bias that were None
    and for dh0 without ``want_dh0``."""
    dev, (B, T, Dn, G, N), st = _ssm_inputs(x, dt, A, Bm, Cm, D, z, dt_bias, 2)
    if h0 is not None:
        _whole("h0", h0, torch.float32, (B, Dn, N), dev)
    _first("dout", dout, 3)
    _like("dout", dout, dout.dtype, (B, T, Dn), dev)
    st += _row_strides("dout", dout, 2)
    if dh_final is not None:
        _whole("dh_final", dh_final, torch.float32, (B, Dn, N), dev)
    code = _dt_of("grad_dtype", grad_dtype)
    dx = _new(dout, grad_dtype, x.shape, dev)
    ddt = torch.empty_like(dx)
    dz = None if z is None else torch.empty_like(dx)
    dB = _new(Bm, grad_dtype, Bm.shape, dev)
    dC = torch.empty_like(dB)
    if Dn == 0:             # sums over no channels, which the C call leaves alone
        dB.zero_()
        dC.zero_()
    dA = torch.empty_like(A)
    dD = None if D is None else torch.empty_like(D)
    db = None if dt_bias is None else torch.empty_like(dt_bias)
    dh0 = _new(dh_final, torch.float32, (B, Dn, N), dev) if want_dh0 else None
    workspace = _scratch(workspace, _need("gdr_ssm_scan_bwd_workspace_size", B, T, Dn, G, N),
                         dev)
    _run("gdr_ssm_scan_bwd", lib.gdr_ssm_scan_bwd(
        B, T, Dn, G, N, _DT[x.dtype], _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D), _p(z),
        _p(dt_bias), _p(h0), _DT[dout.dtype], _p(dout), _p(dh_final), _i64s(*st),
        GDR_SSM_SOFTPLUS if softplus else 0, code, _p(dx), _p(ddt), _p(dA), _p(dB), _p(dC),
        _p(dD), _p(dz), _p(db), _p(dh0), _p(workspace), workspace.numel(), _raw_stream(dev.index)))
    return dx, ddt, dA, dB, dC, dD, dz, db, dh0


def _as_rows(name, t):
    """[..., C] as rows of C channels one stride apart: (rows, C, stride)."""
    if t.dim() < 1:
        raise ValueError(f"{name} must be [..., C]")
    C = t.shape[-1]
    if t.dim() == 2:
        _row_strides(name, t, 1)
        return t.shape[0], C, t.stride(0)
    if t.is_contiguous():
        return (t.numel() // C if C else 0), C, C
    try:
        v = t.view(-1, C)
    except RuntimeError:
        raise ValueError(f"{name} must be rows one stride apart") from None
    _row_strides(name, v, 1)
    return v.shape[0], C, v.stride(0)


@_on_own_device
def gdr_layer_norm_fwd(x, w=None, b=None, eps=1e-5, *, residual=None, out_dtype=None, y=None,
                       h=None, stream=None):
    """Layer norm over the last axis of x [..., C] (fp32 or bf16), after adding
    ``residual`` (its own dtype) when given.  w, b [C] fp32 or None (ones,
    zeros).  Returns y, or (y, h) with the sum h in the residual's dtype.  x and
    residual may be row slices (one stride from row to row); ``y`` may be x and
    ``h`` may be residual itself."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = _first("x", x, x.dim())
    R, C, xr = _as_rows("x", x)
    rdt, rr = x.dtype, 0
    if residual is not None:
        _first("residual", residual, x.dim())
        _like("residual", residual, residual.dtype, x.shape, dev)
        rdt, rr = residual.dtype, _as_rows("residual", residual)[2]
    elif h is not None:
        raise ValueError("h needs a residual")
    if w is not None:
        _whole("w", w, torch.float32, (C,), dev)
    if b is not None:
        _whole("b", b, torch.float32, (C,), dev)
    odt = out_dtype or (x.dtype if y is None else y.dtype)
    code = _dt_of("output dtype", odt)
    y = _buffer("y", y, odt, x.shape, dev, x)
    if residual is not None:
        h = _buffer("h", h, rdt, x.shape, dev, residual)
    _run("gdr_layer_norm_fwd", lib.gdr_layer_norm_fwd(
        R, C, _DT[x.dtype], _p(x), xr, _DT[rdt], _p(residual), rr, _p(w), _p(b), float(eps),
        code, _p(y), _p(h), _raw_stream(dev.index)))
    return y if residual is None else (y, h)


def gdr_layer_norm_bwd_workspace_size(R, C) -> int:
    """Bytes of device workspace gdr_layer_norm_bwd needs for dw and db."""
    return int(lib.gdr_layer_norm_bwd_workspace_size(R, C))


@_on_own_device
def gdr_layer_norm_bwd(x, w, dy, eps=1e-5, *, dres=None, grad_dtype=torch.float32, want_dw=True,
                       workspace=None, stream=None):
    """Reverse mode of gdr_layer_norm_fwd: x [..., C] is the normalised tensor
    (h where a residual was added), dy [..., C] the gradient of y (fp32 or
    bf16), ``dres`` [..., C] in ``grad_dtype`` or None the gradient that reaches
    x past the norm.  Returns (dx in ``grad_dtype``, dw, db [C] fp32), dw and db
    None without ``want_dw``."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = _first("x", x, x.dim())
    R, C, xr = _as_rows("x", x)
    _first("dy", dy, x.dim())
    _like("dy", dy, dy.dtype, x.shape, dev)
    yr = _as_rows("dy", dy)[2]
    code, rr = _dt_of("grad_dtype", grad_dtype), 0
    if dres is not None:
        _like("dres", dres, grad_dtype, x.shape, dev)
        rr = _as_rows("dres", dres)[2]
    if w is not None:
        _whole("w", w, torch.float32, (C,), dev)
    dx = _new(dy, grad_dtype, x.shape, dev)
    dw = _new(w, torch.float32, (C,), dev) if want_dw else None
    db = torch.empty_like(dw) if want_dw else None
    if want_dw or workspace is not None:
        workspace = _scratch(workspace, _need("gdr_layer_norm_bwd_workspace_size", R, C), dev)
    _run("gdr_layer_norm_bwd", lib.gdr_layer_norm_bwd(
        R, C, _DT[x.dtype], _p(x), xr, _p(w), _DT[dy.dtype], _p(dy), yr, float(eps), code,
        _p(dres), rr, _p(dx), _p(dw), _p(db), _p(workspace),
        0 if workspace is None else workspace.numel(), _raw_stream(dev.index)))
    return dx, dw, db
