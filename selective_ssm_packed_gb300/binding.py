"""Thin ctypes binding of libvarlen_ssm.so (argument marshalling only).

Each function carries the name of the C entry point it calls (see
include/varlen_ssm.h for the definitions, layouts and error behaviour).  It
checks that the torch tensors it is handed are contiguous CUDA tensors of the
right dtype, allocates outputs and workspaces the caller did not pass (with
torch, i.e. the caching allocator), passes raw device pointers and torch's
current stream, and raises VssmError on a non-zero status.  All arithmetic
happens in the library's CUDA kernels; if the library is missing, every call
raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

VSSM_F32, VSSM_BF16 = 0, 1
VSSM_STATE_CHUNK = 32
VSSM_DBG_DROP_FLAG, VSSM_DBG_WAIT_NS, VSSM_DBG_DELAY_ITEM, VSSM_DBG_DELAY_NS = 1, 2, 3, 4
VSSM_DBG_FORCE_COPY_TIMEOUT, VSSM_DBG_CHECK_FINITE, VSSM_DBG_KERNEL_EVENTS = 5, 6, 7
# the call kinds vssm_kernel_time reports
KERNEL_KINDS = {"conv_fwd": 0, "scan_fwd": 1, "scan_bwd": 2, "conv_bwd": 3}
ERR = {0: "VSSM_OK", -1: "VSSM_ERR_ARG", -2: "VSSM_ERR_DTYPE", -3: "VSSM_ERR_ALIGN",
       -4: "VSSM_ERR_WORKSPACE", -5: "VSSM_ERR_CUDA", -6: "VSSM_ERR_UNSUPPORTED",
       -16: "VSSM_ERR_BAD_CU_SEQLENS", -17: "VSSM_ERR_LOOKBACK_TIMEOUT", -18: "VSSM_ERR_NONFINITE",
       -19: "VSSM_ERR_DEVICE_CHECK", -20: "VSSM_ERR_BAD_INDEX",
       -21: "VSSM_ERR_BAD_SAVED"}

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_f32 = ctypes.c_float

# name -> (restype, argtypes)
SIGNATURES = {
    "varlen_position_indices": (ctypes.c_int, [_vp, _i32, _i64, _vp, _vp, _vp]),
    "vssm_status_code": (ctypes.c_int, [_i32]),
    "varlen_conv1d_fwd_workspace_size": (_sz, [_i64, _i32, _i32]),
    "varlen_conv1d_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                                         ctypes.c_int, _vp, _vp, _vp, _vp, _sz, _vp]),
    "varlen_conv1d_bwd_workspace_size": (_sz, [_i64, _i32, _i32]),
    "varlen_conv1d_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                                         ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "varlen_selective_scan_fwd_workspace_size": (_sz, [_i64, _i32, _i32]),
    "varlen_selective_scan_chunk_states_size": (_sz, [_i64, _i32, _i32]),
    "varlen_selective_scan_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                                 ctypes.c_float, _i32,
                                                 _vp, _vp, _i32, _i64, _i32, _i32, ctypes.c_int,
                                                 _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "varlen_conv1d_scan_fwd": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _i32, ctypes.c_float, _i32,
                                              _vp, _vp, _i32, _i64, _i32, _i32, ctypes.c_int,
                                              _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "varlen_selective_scan_bwd_workspace_size": (_sz, [_i64, _i32, _i32]),
    "varlen_selective_scan_bwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                                 ctypes.c_float, _i32, _vp,
                                                 _vp, _vp, _i32, _i64, _i32, _i32, ctypes.c_int, _vp,
                                                 _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                 _vp, _vp, _sz, _vp]),
    "varlen_selective_scan_fwd_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                                         ctypes.c_float, _i32,
                                                         _vp, _vp, _i32, _i64, _i32, _i32, ctypes.c_int,
                                                         _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "varlen_qk_norm_rope_fwd": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32,
                                               _i32, _i32, _i32, _f32, ctypes.c_int, _vp, _vp, _vp, _vp]),
    "varlen_qk_norm_rope_bwd_workspace_size": (_sz, [_i32]),
    "varlen_qk_norm_rope_bwd": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _i64,
                                               _i32, _i32, _i32, _i32, _i32, _f32, ctypes.c_int, _vp, _vp, _vp, _vp,
                                               _vp, _sz, _vp]),
    "varlen_gated_delta_saved_size": (_sz, [_i64, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "varlen_gated_delta_fwd_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "varlen_gated_delta_bwd_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "vssm_gated_delta_walks": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "varlen_gated_delta_fwd": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _i32, _i64, _i32,
                                              _i32, _i32, _i32, ctypes.c_int, _vp, _vp, _vp, _vp, _sz, _vp, _sz, _vp]),
    "varlen_gated_delta_bwd": (ctypes.c_int, [_vp, _f32, _vp, _i32, _i64, _i32, _i32, _i32, _i32, ctypes.c_int, _vp,
                                              _sz, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "varlen_gated_delta_step": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _vp, _i64, _i64,
                                               _i32, _i32, _i32, _i32, ctypes.c_int, _vp, _vp, _vp]),
    "varlen_linear_attn_fwd_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "varlen_linear_attn_bwd_workspace_size": (_sz, [_i64, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "vssm_linear_attn_segment": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, _i32, ctypes.c_int, _i32]),
    "varlen_linear_attn_fwd": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _f32, _vp, _i32, _i64, _i32,
                                              _i32, _i32, _i32, ctypes.c_int, _vp, _vp, _vp, _vp, _sz, _vp]),
    "varlen_linear_attn_bwd": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _vp, _f32, _vp, _i32, _i64,
                                              _i32, _i32, _i32, _i32, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _vp, _sz, _vp]),
    "varlen_linear_attn_step": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _f32, _vp, _vp, _i64, _i64,
                                               _i32, _i32, _i32, _i32, ctypes.c_int, _vp, _vp, _vp]),
    "varlen_layer_norm_fwd": (ctypes.c_int, [_vp, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _f32, ctypes.c_int, _vp, _vp,
                                             _vp]),
    "varlen_layer_norm_bwd_workspace_size": (_sz, [_i64, _i32, _i32]),
    "varlen_layer_norm_bwd": (ctypes.c_int, [_vp, _i64, _i32, _vp, _vp, _vp, _i64, _i32, _i32, _f32, ctypes.c_int, _vp,
                                             _vp, _vp, _vp, _vp, _sz, _vp]),
    "varlen_pack_sequences": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _vp,
                                             ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_double)]),
    "vssm_read_status": (ctypes.c_int, [_vp, _vp, ctypes.POINTER(ctypes.c_int)]),
    "vssm_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "vssm_last_error": (ctypes.c_char_p, []),
    "vssm_checks_build": (ctypes.c_int, []),
    "vssm_kernel_time": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_int64)]),
    "vssm_debug_set": (ctypes.c_int, [ctypes.c_int, _i64]),
}

_lib = None


class VssmError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {ERR.get(code, code)} ({code}): {last_error()}")


def library_path() -> str:
    """The library this process loads: the checked build when VSSM_CHECKS=1
    is set in the environment, else the ordinary one."""
    return _build.lib_path()


def lib():
    """The loaded library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first with "
                               "selective_ssm_packed_gb300.build.build()")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def last_error() -> str:
    return lib().vssm_last_error().decode()


def strerror(code: int) -> str:
    return lib().vssm_strerror(code).decode()


def debug_set(knob: int, value: int) -> None:
    _check(lib().vssm_debug_set(knob, value), "vssm_debug_set")


def _check(rc, what):
    if rc != 0:
        raise VssmError(rc, what)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return VSSM_F32
    if t.dtype == torch.bfloat16:
        return VSSM_BF16
    raise TypeError(f"I/O tensors must be float32 or bfloat16, got {t.dtype}")


def _ptr(t, name, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr() or None


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ws(workspace, nbytes, device):
    if workspace is None:
        return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace too small: {workspace.numel()} < {nbytes} bytes")
    return workspace


def read_status(workspace: torch.Tensor, stream=None) -> int:
    st = ctypes.c_int(0)
    _check(lib().vssm_read_status(_ptr(workspace, "workspace"), _stream(stream), ctypes.byref(st)),
           "vssm_read_status")
    return st.value


def kernel_time(kind: str):
    """(total ms, launches) of one kind of call's main kernel since the last
    read, from the events VSSM_DBG_KERNEL_EVENTS records."""
    ms, n = ctypes.c_double(0.0), ctypes.c_int64(0)
    _check(lib().vssm_kernel_time(KERNEL_KINDS[kind], ctypes.byref(ms), ctypes.byref(n)), "vssm_kernel_time")
    return ms.value, n.value


def status_code(word: int) -> int:
    return lib().vssm_status_code(int(word))


# ------------------------------------------------------------------ position indices
def varlen_position_indices(cu_seqlens, total_tokens, out=None, status=None, stream=None):
    cu = cu_seqlens
    _ptr(cu, "cu_seqlens", torch.int32)
    T = int(total_tokens)
    if out is None:
        out = torch.empty(T, dtype=torch.int32, device=cu.device)
    _check(lib().varlen_position_indices(_ptr(cu, "cu_seqlens"), cu.numel() - 1, T,
                                         _ptr(out, "out", torch.int32),
                                         _ptr(status, "status", torch.int32), _stream(stream)),
           "varlen_position_indices")
    return out


# ------------------------------------------------------------------ conv1d
def conv1d_fwd_workspace_size(T, D, W):
    return lib().varlen_conv1d_fwd_workspace_size(int(T), int(D), int(W))


def conv1d_bwd_workspace_size(T, D, W):
    return lib().varlen_conv1d_bwd_workspace_size(int(T), int(D), int(W))


def varlen_conv1d_fwd(x, weight, bias, cu_seqlens, position_indices=None, apply_silu=True,
                      out=None, workspace=None, stream=None, x_init=None, x_last=None):
    """Returns u, or (u, x_last) when x_last is asked for (True allocates,
    a tensor is filled).  x_init: (S, D, W-1) f32 inputs before each sequence
    (a cut sequence's previous part's x_last); None: the plain early stop."""
    T, D = x.shape
    W = weight.shape[1]
    out = torch.empty_like(x) if out is None else out
    want_last = x_last is not None and x_last is not False
    if x_last is True:
        x_last = torch.empty((cu_seqlens.numel() - 1, D, W - 1), dtype=torch.float32, device=x.device)
    elif x_last is False:
        x_last = None
    ws = _ws(workspace, conv1d_fwd_workspace_size(T, D, W), x.device)
    _check(lib().varlen_conv1d_fwd(
        _ptr(x, "x"), _ptr(weight, "weight", torch.float32), _ptr(bias, "bias", torch.float32),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), _ptr(position_indices, "position_indices", torch.int32),
        cu_seqlens.numel() - 1, T, D, W, int(bool(apply_silu)), _dt(x), _ptr(out, "out", x.dtype),
        _ptr(x_init, "x_init", torch.float32), _ptr(x_last, "x_last", torch.float32),
        _ptr(ws, "workspace"), ws.numel(), _stream(stream)), "varlen_conv1d_fwd")
    return (out, x_last) if want_last else out


def varlen_conv1d_bwd(x, weight, bias, du, cu_seqlens, position_indices=None, apply_silu=True,
                      dx=None, dweight=None, dbias=None, workspace=None, stream=None, x_init=None,
                      dx_last=None, dx_init=None):
    """Returns (dx, dweight, dbias), and dx_init last when it is asked for
    (True allocates, a tensor is filled).  x_init: the forward call's;
    dx_last: (S, D, W-1) gradient reaching each sequence's x_last."""
    T, D = x.shape
    W = weight.shape[1]
    dx = torch.empty_like(x) if dx is None else dx
    dweight = torch.empty_like(weight) if dweight is None else dweight
    if dbias is None and bias is not None:
        dbias = torch.empty_like(bias)
    want_init = dx_init is not None and dx_init is not False
    if dx_init is True:
        dx_init = torch.empty((cu_seqlens.numel() - 1, D, W - 1), dtype=torch.float32, device=x.device)
    elif dx_init is False:
        dx_init = None
    ws = _ws(workspace, conv1d_bwd_workspace_size(T, D, W), x.device)
    _check(lib().varlen_conv1d_bwd(
        _ptr(x, "x"), _ptr(weight, "weight", torch.float32), _ptr(bias, "bias", torch.float32),
        _ptr(du, "du", x.dtype), _ptr(cu_seqlens, "cu_seqlens", torch.int32),
        _ptr(position_indices, "position_indices", torch.int32), cu_seqlens.numel() - 1, T, D, W,
        int(bool(apply_silu)), _dt(x), _ptr(dx, "dx", x.dtype), _ptr(dweight, "dweight", torch.float32),
        _ptr(dbias, "dbias", torch.float32), _ptr(x_init, "x_init", torch.float32),
        _ptr(dx_last, "dx_last", torch.float32), _ptr(dx_init, "dx_init", torch.float32),
        _ptr(ws, "workspace"), ws.numel(), _stream(stream)),
        "varlen_conv1d_bwd")
    return (dx, dweight, dbias, dx_init) if want_init else (dx, dweight, dbias)


# ------------------------------------------------------------------ selective scan
def scan_fwd_workspace_size(T, D, N):
    return lib().varlen_selective_scan_fwd_workspace_size(int(T), int(D), int(N))


def scan_bwd_workspace_size(T, D, N):
    return lib().varlen_selective_scan_bwd_workspace_size(int(T), int(D), int(N))


def chunk_states_shape(T, D, N):
    return ((int(T) + VSSM_STATE_CHUNK - 1) // VSSM_STATE_CHUNK, int(N), int(D))


def varlen_selective_scan_fwd(u, delta_raw, A, B, C, Dskip, z, dt_bias, cu_seqlens,
                              position_indices=None, delta_softplus=True, out=None,
                              chunk_states=True, workspace=None, stream=None, y=None, gate_floor=0.0,
                              a_log=False, initial_states=None, final_states=None):
    """Returns (out, chunk_states), or (out, chunk_states, y) when y is asked
    for.  chunk_states=True allocates the saved-state array the backward call
    needs, False/None skips it, a tensor is filled.  y (the output before the
    gate, which the backward call can take for dz): None/False skips it, True
    allocates it, a tensor is filled.  gate_floor: the GateFloor gate
    SiLU(z) + gate_floor; a_log: A holds A_log (A = -exp(A_log)).
    initial_states: (S, D, N) f32 state each sequence starts from (None: zero).
    final_states: None skips them, True allocates, a tensor is filled; when
    asked for they come last in the returned tuple."""
    T, D = u.shape
    N = A.shape[1]
    out = torch.empty_like(u) if out is None else out
    want_y = y is not None and y is not False
    if y is True:
        y = torch.empty_like(u)
    elif y is False:
        y = None
    S = cu_seqlens.numel() - 1
    want_final = final_states is not None and final_states is not False
    if final_states is True:
        final_states = torch.empty((S, D, N), dtype=torch.float32, device=u.device)
    elif final_states is False:
        final_states = None
    if chunk_states is True:
        chunk_states = torch.empty(chunk_states_shape(T, D, N), dtype=torch.float32, device=u.device)
    elif chunk_states is False:
        chunk_states = None
    ws = _ws(workspace, scan_fwd_workspace_size(T, D, N), u.device)
    dt = u.dtype
    _check(lib().varlen_selective_scan_fwd(
        _ptr(u, "u"), _ptr(delta_raw, "delta_raw", dt), _ptr(A, "A", torch.float32),
        _ptr(B, "B", dt), _ptr(C, "C", dt), _ptr(Dskip, "Dskip", torch.float32), _ptr(z, "z", dt),
        _ptr(dt_bias, "dt_bias", torch.float32), int(bool(delta_softplus)), float(gate_floor),
        int(bool(a_log)),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), _ptr(position_indices, "position_indices", torch.int32),
        cu_seqlens.numel() - 1, T, D, N, _dt(u), _ptr(out, "out", dt), _ptr(y, "y", dt),
        _ptr(chunk_states, "chunk_states", torch.float32),
        _ptr(initial_states, "initial_states", torch.float32), _ptr(final_states, "final_states", torch.float32),
        _ptr(ws, "workspace"), ws.numel(), _stream(stream)), "varlen_selective_scan_fwd")
    res = (out, chunk_states) + ((y,) if want_y else ()) + ((final_states,) if want_final else ())
    return res


def varlen_conv1d_scan_fwd(x, conv_weight, conv_bias, delta_raw, A, B, C, Dskip, z, dt_bias, cu_seqlens,
                           position_indices=None, apply_silu=True, delta_softplus=True, u=True, out=None,
                           chunk_states=True, workspace=None, stream=None, y=None, gate_floor=0.0,
                           a_log=False, initial_states=None, final_states=None):
    """The conv1d forward and the selective-scan forward in one call (u computed
    on chip; results equal the two calls' bit for bit).  Returns (u, out,
    chunk_states) plus y and final_states when asked for, as
    varlen_selective_scan_fwd; u: True allocates the conv output (the backward
    needs it), None/False skips writing it, a tensor is filled."""
    T, D = x.shape
    N = A.shape[1]
    W = conv_weight.shape[1]
    out = torch.empty_like(x) if out is None else out
    if u is True:
        u = torch.empty_like(x)
    elif u is False:
        u = None
    want_y = y is not None and y is not False
    if y is True:
        y = torch.empty_like(x)
    elif y is False:
        y = None
    S = cu_seqlens.numel() - 1
    want_final = final_states is not None and final_states is not False
    if final_states is True:
        final_states = torch.empty((S, D, N), dtype=torch.float32, device=x.device)
    elif final_states is False:
        final_states = None
    if chunk_states is True:
        chunk_states = torch.empty(chunk_states_shape(T, D, N), dtype=torch.float32, device=x.device)
    elif chunk_states is False:
        chunk_states = None
    ws = _ws(workspace, scan_fwd_workspace_size(T, D, N), x.device)
    dt = x.dtype
    _check(lib().varlen_conv1d_scan_fwd(
        _ptr(x, "x"), _ptr(conv_weight, "conv_weight", torch.float32), _ptr(conv_bias, "conv_bias", torch.float32),
        W, int(bool(apply_silu)), _ptr(delta_raw, "delta_raw", dt), _ptr(A, "A", torch.float32),
        _ptr(B, "B", dt), _ptr(C, "C", dt), _ptr(Dskip, "Dskip", torch.float32), _ptr(z, "z", dt),
        _ptr(dt_bias, "dt_bias", torch.float32), int(bool(delta_softplus)), float(gate_floor), int(bool(a_log)),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), _ptr(position_indices, "position_indices", torch.int32),
        cu_seqlens.numel() - 1, T, D, N, _dt(x), _ptr(u, "u", dt), _ptr(out, "out", dt), _ptr(y, "y", dt),
        _ptr(chunk_states, "chunk_states", torch.float32),
        _ptr(initial_states, "initial_states", torch.float32), _ptr(final_states, "final_states", torch.float32),
        _ptr(ws, "workspace"), ws.numel(), _stream(stream)), "varlen_conv1d_scan_fwd")
    return (u, out, chunk_states) + ((y,) if want_y else ()) + ((final_states,) if want_final else ())


def varlen_selective_scan_bwd(u, delta_raw, A, B, C, Dskip, z, dt_bias, dout, cu_seqlens,
                              chunk_states, position_indices=None, delta_softplus=True,
                              grads=None, workspace=None, stream=None, y=None, gate_floor=0.0,
                              a_log=False, initial_states=None, d_final_states=None,
                              d_initial_states=None):
    """Returns dict du, ddelta_raw, dA, dB, dC, dDskip, dz, d_dt_bias.  y: the
    forward call's pre-gate output (optional; dz then reads it instead of
    recomputing it).  gate_floor, a_log: as in the forward call; with a_log
    the dA entry holds dA_log = dA * A.  initial_states: the forward call's;
    d_final_states: (S, D, N) gradient reaching each sequence's final state;
    d_initial_states: True allocates (or a tensor to fill) the gradient
    reaching each sequence's starting state, returned as "d_initial_states"."""
    T, D = u.shape
    N = A.shape[1]
    dt = u.dtype
    g = dict(grads or {})
    # outputs the caller did not pass are allocated here (only those)
    make = {"du": lambda: torch.empty_like(u), "ddelta_raw": lambda: torch.empty_like(u),
            "dA": lambda: torch.empty_like(A),
            "dB": lambda: torch.empty((T, N), dtype=torch.float32, device=u.device),
            "dC": lambda: torch.empty((T, N), dtype=torch.float32, device=u.device),
            "dDskip": lambda: torch.empty_like(Dskip) if Dskip is not None else None,
            "dz": lambda: torch.empty_like(z) if z is not None else None,
            "d_dt_bias": lambda: torch.empty_like(dt_bias) if dt_bias is not None else None}
    for k, f in make.items():
        if k not in g:
            g[k] = f()
    if d_initial_states is True:
        d_initial_states = torch.empty((cu_seqlens.numel() - 1, D, N), dtype=torch.float32, device=u.device)
    elif d_initial_states is False:
        d_initial_states = None
    g["d_initial_states"] = d_initial_states
    ws = _ws(workspace, scan_bwd_workspace_size(T, D, N), u.device)
    _check(lib().varlen_selective_scan_bwd(
        _ptr(u, "u"), _ptr(delta_raw, "delta_raw", dt), _ptr(A, "A", torch.float32),
        _ptr(B, "B", dt), _ptr(C, "C", dt), _ptr(Dskip, "Dskip", torch.float32), _ptr(z, "z", dt),
        _ptr(dt_bias, "dt_bias", torch.float32), int(bool(delta_softplus)), float(gate_floor),
        int(bool(a_log)), _ptr(dout, "dout", dt),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), _ptr(position_indices, "position_indices", torch.int32),
        cu_seqlens.numel() - 1, T, D, N, _dt(u), _ptr(chunk_states, "chunk_states", torch.float32),
        _ptr(y, "y", dt), _ptr(initial_states, "initial_states", torch.float32),
        _ptr(d_final_states, "d_final_states", torch.float32),
        _ptr(d_initial_states, "d_initial_states", torch.float32), _ptr(g["du"], "du", dt), _ptr(g["ddelta_raw"], "ddelta_raw", dt),
        _ptr(g["dA"], "dA", torch.float32), _ptr(g["dB"], "dB", torch.float32),
        _ptr(g["dC"], "dC", torch.float32), _ptr(g["dDskip"], "dDskip", torch.float32),
        _ptr(g["dz"], "dz", dt), _ptr(g["d_dt_bias"], "d_dt_bias", torch.float32),
        _ptr(ws, "workspace"), ws.numel(), _stream(stream)), "varlen_selective_scan_bwd")
    return g


# ------------------------------------------------------------------ heads of a token
def _heads(t, name, dtype=None, heads=None, width=None):
    """(pointer, token stride) of a (T, H, K) CUDA tensor whose heads are
    contiguous and whose tokens may be any distance apart."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be (tokens, heads, width), got {tuple(shape)}")
    T, H, K = shape
    if (heads is not None and H != heads) or (width is not None and K != width):
        raise ValueError(f"{name} must be (tokens, {heads or H}, {width or K}), got {tuple(shape)}")
    along, across, inner = t.stride()
    if ((K > 1 and inner != 1) or (H > 1 and across != K)) and t.numel():
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr() or None, (along if T > 1 else H * K)


def _shaped(t, name, shape, dtype=torch.float32):
    """_ptr of a tensor of the given shape."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or None


def _stream_of(t, stream):
    """The raw handle of `stream`, or of the current stream of t's device
    (looked up without building a torch.cuda.Stream, which takes longer than
    a launch)."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(t.get_device())


def _new(shape, dtype, like, stream):
    """Memory on like's device that belongs to the stream the call runs on, so
    that it can neither still be in use by another one nor go back to it
    before the call's kernels are through."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _result(t, name, like, stream):
    """(tensor, pointer) of a result of like's shape and type: t, looked over,
    or new memory, as _new's."""
    if t is not None:
        return t, _shaped(t, name, like.shape, like.dtype)
    if stream is None:
        t = torch.empty_like(like, memory_format=torch.contiguous_format)
    else:
        t = _new(like.shape, like.dtype, like, stream)
    return t, t.data_ptr() or None


def _room(workspace, nbytes, like, stream):
    """_ws, new memory being the call's stream's."""
    if workspace is None:
        return _new((max(int(nbytes), 16),), torch.uint8, like, stream)
    return _ws(workspace, nbytes, like.device)


def _asked(t, shape, like, stream):
    """f32 result; None / False: not wanted; True: allocated; a tensor: filled."""
    if t is None or t is False:
        return None
    return _new(shape, torch.float32, like, stream) if t is True else t


# ------------------------------------------------------------------ norm and rotation of queries and keys
QK_NORM_MODES = {"rms": 0, "l2": 1}


def _norm_args(q, k, q_weight, k_weight, cos, sin, positions, mode):
    if mode not in QK_NORM_MODES:
        raise ValueError(f"mode must be one of {sorted(QK_NORM_MODES)}, got {mode!r}")
    qp, sq = _heads(q, "q")
    T, Hq, K = q.shape
    kp, sk = _heads(k, "k", q.dtype, width=K)
    Hk = k.shape[1]
    if k.shape[0] != T:
        raise ValueError(f"q has {T} tokens, k has {k.shape[0]}")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin must be given together")
    rows = half = 0
    if cos is not None:
        rows, half = cos.shape
        if positions is None:
            raise ValueError("a rotation needs positions")
    return [qp, kp, sq, sk, _shaped(q_weight, "q_weight", (K,)), _shaped(k_weight, "k_weight", (K,)),
            _ptr(cos, "cos", torch.float32), _shaped(sin, "sin", (rows, half)),
            _shaped(positions, "positions", (T,), torch.int32) if cos is not None else None, rows], (T, Hq, Hk, K, 2 * half)


def varlen_qk_norm_rope_fwd(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, mode="rms",
                            eps=1e-6, q_out=None, k_out=None, status=None, stream=None):
    """Returns (q_out, k_out): each head of q (T, Hq, K) and k (T, Hk, K)
    normalised (mode "rms" or "l2"), scaled by its weight (K) and rotated by
    its token's position with the tables cos, sin (P, rot / 2); cos None: no
    rotation.  q and k may be slices of wider rows (heads contiguous).
    status: optional int32 tensor for positions outside the tables."""
    lead, (T, Hq, Hk, K, rot) = _norm_args(q, k, q_weight, k_weight, cos, sin, positions, mode)
    q_out, qp = _result(q_out, "q_out", q, stream)
    k_out, kp = _result(k_out, "k_out", k, stream)
    _check(lib().varlen_qk_norm_rope_fwd(
        *lead, T, Hq, Hk, K, rot, QK_NORM_MODES[mode], float(eps), _dt(q), qp, kp, _ptr(status, "status", torch.int32),
        _stream_of(q, stream)), "varlen_qk_norm_rope_fwd")
    return q_out, k_out


def varlen_qk_norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, mode="rms", eps=1e-6,
                            grads=None, workspace=None, stream=None):
    """Returns dict dq, dk and, where the forward call had weights, dq_weight,
    dk_weight (else None); grads: tensors to fill instead, by those names."""
    lead, (T, Hq, Hk, K, rot) = _norm_args(q, k, q_weight, k_weight, cos, sin, positions, mode)
    g = dict(grads or {})
    make = {"dq": ((T, Hq, K), q.dtype), "dk": ((T, Hk, K), q.dtype), "dq_weight": ((K,), torch.float32),
            "dk_weight": ((K,), torch.float32)}
    for n, w in (("dq", q), ("dk", k), ("dq_weight", q_weight), ("dk_weight", k_weight)):
        if n not in g:
            g[n] = _new(*make[n], q, stream) if w is not None else None
    ws = _room(workspace, lib().varlen_qk_norm_rope_bwd_workspace_size(K), q, stream)
    _check(lib().varlen_qk_norm_rope_bwd(
        *lead, _shaped(dq_out, "dq_out", (T, Hq, K), q.dtype), _shaped(dk_out, "dk_out", (T, Hk, K), q.dtype),
        T, Hq, Hk, K, rot, QK_NORM_MODES[mode], float(eps), _dt(q), *(_shaped(g[n], n, *make[n]) for n in make),
        _ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream_of(q, stream)), "varlen_qk_norm_rope_bwd")
    return g


# ------------------------------------------------------------------ gated delta rule
def gated_delta_saved_size(T, S, Hk, Hv, K, V, dtype):
    return lib().varlen_gated_delta_saved_size(int(T), int(S), int(Hk), int(Hv), int(K), int(V), int(dtype))


def gated_delta_fwd_workspace_size(T, S, Hk, Hv, K, V, dtype):
    return lib().varlen_gated_delta_fwd_workspace_size(int(T), int(S), int(Hk), int(Hv), int(K), int(V), int(dtype))


def gated_delta_bwd_workspace_size(T, S, Hk, Hv, K, V, dtype):
    return lib().varlen_gated_delta_bwd_workspace_size(int(T), int(S), int(Hk), int(Hv), int(K), int(V), int(dtype))


def gated_delta_walks(T, S, Hk, Hv, K, V, dtype):
    return lib().vssm_gated_delta_walks(int(T), int(S), int(Hk), int(Hv), int(K), int(V), int(dtype))


def _delta_args(q, k, v, g, beta):
    qp, sq = _heads(q, "q")
    T, Hk, K = q.shape
    kp, sk = _heads(k, "k", q.dtype, Hk, K)
    vp, sv = _heads(v, "v", q.dtype)
    _, Hv, V = v.shape
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError(f"q, k and v have {T}, {k.shape[0]} and {v.shape[0]} tokens")
    return [qp, kp, vp, sq, sk, sv, _shaped(g, "g", (T, Hv)), _shaped(beta, "beta", (T, Hv))], (T, Hk, Hv, K, V)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t


def _num_seqs(cu_seqlens):
    S = _cuda(cu_seqlens, "cu_seqlens").numel() - 1
    if S < 0:
        raise ValueError("cu_seqlens must have at least one entry")
    return S


def varlen_gated_delta_fwd(q, k, v, g, beta, cu_seqlens, scale=None, out=None, saved=True, workspace=None, stream=None,
                           initial_states=None, final_states=None):
    """Returns (out, saved), and final_states last when they are asked for.
    q, k (T, Hk, K), v (T, Hv, V) may be slices of wider rows; g, beta (T, Hv)
    f32; scale: K ** -0.5 when None.  saved=True allocates the array the
    backward call needs (None / False: not written, None returned), a uint8
    tensor is filled.  initial_states, final_states: (S, Hv, K, V) f32, the
    latter None / False, True or a tensor to fill."""
    args, (T, Hk, Hv, K, V) = _delta_args(q, k, v, g, beta)
    S, dt = _num_seqs(cu_seqlens), _dt(q)
    sizes = (T, S, Hk, Hv, K, V, dt)
    out, op = _result(out, "out", v, stream)
    want_final = final_states is not None and final_states is not False
    final_states = _asked(final_states, (S, Hv, K, V), q, stream)
    if saved is True:
        saved = _new((max(gated_delta_saved_size(*sizes), 16),), torch.uint8, q, stream)
    elif saved is False:
        saved = None
    ws = _room(workspace, 256 if saved is not None else gated_delta_fwd_workspace_size(*sizes), q, stream)
    _check(lib().varlen_gated_delta_fwd(
        *args, float(K ** -0.5 if scale is None else scale), _ptr(cu_seqlens, "cu_seqlens", torch.int32), S, T, Hk, Hv,
        K, V, dt, op, _shaped(initial_states, "initial_states", (S, Hv, K, V)),
        _shaped(final_states, "final_states", (S, Hv, K, V)), _ptr(saved, "saved", torch.uint8),
        saved.numel() if saved is not None else 0, _ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream_of(q, stream)),
        "varlen_gated_delta_fwd")
    return (out, saved) + ((final_states,) if want_final else ())


def varlen_gated_delta_bwd(q, k, v, g, beta, dout, cu_seqlens, saved, scale=None, grads=None, workspace=None,
                           stream=None, d_final_states=None, d_initial_states=None):
    """Returns dict dq, dk, dv, dg, dbeta, d_initial_states.  The inputs, scale
    and saved are the forward call's (saved holds what the gradients need of
    q .. beta: only their shapes are read).  d_final_states: (S, Hv, K, V) f32,
    the gradient reaching the final states; d_initial_states: None / False,
    True or a tensor to fill.  grads: tensors to fill, by name."""
    _, (T, Hk, Hv, K, V) = _delta_args(q, k, v, g, beta)
    S, dt = _num_seqs(cu_seqlens), _dt(q)
    sizes = (T, S, Hk, Hv, K, V, dt)
    _cuda(saved, "saved (the forward call's array)")
    r = dict(grads or {})
    shapes = {"dq": ((T, Hk, K), q.dtype), "dk": ((T, Hk, K), q.dtype), "dv": ((T, Hv, V), q.dtype),
              "dg": ((T, Hv), torch.float32), "dbeta": ((T, Hv), torch.float32)}
    for n, (shape, d) in shapes.items():
        if n not in r:
            r[n] = _new(shape, d, q, stream)
    r["d_initial_states"] = _asked(d_initial_states, (S, Hv, K, V), q, stream)
    ws = _room(workspace, gated_delta_bwd_workspace_size(*sizes), q, stream)
    _check(lib().varlen_gated_delta_bwd(
        _shaped(dout, "dout", (T, Hv, V), q.dtype), float(K ** -0.5 if scale is None else scale),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), S, T, Hk, Hv, K, V, dt, _ptr(saved, "saved", torch.uint8),
        saved.numel(), _shaped(d_final_states, "d_final_states", (S, Hv, K, V)),
        _shaped(r["d_initial_states"], "d_initial_states", (S, Hv, K, V)),
        *(_shaped(r[n], n, shape, d) for n, (shape, d) in shapes.items()),
        _ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream_of(q, stream)), "varlen_gated_delta_bwd")
    return r


def varlen_gated_delta_step(q, k, v, g, beta, states, state_indices=None, scale=None, out=None, status=None,
                            stream=None):
    """Returns out (B, Hv, V): one token of each of B sequences, q, k (B, Hk, K),
    v (B, Hv, V), g, beta (B, Hv), against states (slots, Hv, K, V) f32, which
    are updated in place.  state_indices: int32 (B) slots, all different,
    negative for a padded entry (None: entry b uses slot b).  status: optional
    int32 tensor for indices outside the pool."""
    args, (B, Hk, Hv, K, V) = _delta_args(q, k, v, g, beta)
    if _cuda(states, "states").dim() != 4:
        raise ValueError(f"states must be (slots, {Hv}, {K}, {V}), got {tuple(states.shape)}")
    slots = states.shape[0]
    out, op = _result(out, "out", v, stream)
    _check(lib().varlen_gated_delta_step(
        *args, float(K ** -0.5 if scale is None else scale), _shaped(states, "states", (slots, Hv, K, V)),
        _shaped(state_indices, "state_indices", (B,), torch.int32), slots, B, Hk, Hv, K, V, _dt(q), op,
        _ptr(status, "status", torch.int32), _stream_of(q, stream)),
        "varlen_gated_delta_step")
    return out


# ------------------------------------------------------------------ linear attention with a decay for each head
class _Here:
    """A context that leaves the current device alone."""

    def __enter__(self):
        return self

    def __exit__(self, *_):
        return False


_HERE = _Here()


def _device_of(t):
    """A context in which t's device is the current one, which the library
    launches on."""
    return _HERE if t.get_device() == torch._C._cuda_getDevice() else torch.cuda.device(t.device)


def _together(first, *others):
    """Refuses tensors on several devices: a kernel would read memory that is
    not its device's."""
    device = first.get_device()
    for t in others:
        if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != device:
            raise ValueError(f"the tensors of a call must be on one device, got {first.device} and {t.device}")


def linear_attn_fwd_workspace_size(T, S, Hk, Hv, K, V, dtype):
    return lib().varlen_linear_attn_fwd_workspace_size(int(T), int(S), int(Hk), int(Hv), int(K), int(V), int(dtype))


def linear_attn_bwd_workspace_size(T, S, Hk, Hv, K, V, dtype):
    return lib().varlen_linear_attn_bwd_workspace_size(int(T), int(S), int(Hk), int(Hv), int(K), int(V), int(dtype))


def linear_attn_segment(T, S, Hk, Hv, K, V, dtype, backward=False):
    return lib().vssm_linear_attn_segment(int(T), int(S), int(Hk), int(Hv), int(K), int(V), int(dtype), int(backward))


def _linear_args(q, k, v, g):
    qp, sq = _heads(q, "q")
    T, Hk, K = q.shape
    kp, sk = _heads(k, "k", q.dtype, Hk, K)
    vp, sv = _heads(v, "v", q.dtype)
    _, Hv, V = v.shape
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError(f"q, k and v have {T}, {k.shape[0]} and {v.shape[0]} tokens")
    per_token = _cuda(g, "g").dim() != 1
    return [qp, kp, vp, sq, sk, sv, _shaped(g, "g", (T, Hv) if per_token else (Hv,)), int(per_token)], (T, Hk, Hv, K, V)


def varlen_linear_attn_fwd(q, k, v, g, cu_seqlens, scale=None, out=None, workspace=None, stream=None,
                           initial_states=None, final_states=None):
    """Returns out, or (out, final_states) when those are asked for.  q, k
    (T, Hk, K), v (T, Hv, V) may be slices of wider rows; g f32 log decays,
    (T, Hv) or one for each head, (Hv); scale: K ** -0.5 when None.
    initial_states, final_states: (S, Hv, K, V) f32, the latter None / False,
    True or a tensor to fill."""
    args, (T, Hk, Hv, K, V) = _linear_args(q, k, v, g)
    S, dt = _num_seqs(cu_seqlens), _dt(q)
    _together(q, k, v, g, cu_seqlens, out, workspace, initial_states, final_states)
    with _device_of(q):
        out, op = _result(out, "out", v, stream)
        want_final = final_states is not None and final_states is not False
        final_states = _asked(final_states, (S, Hv, K, V), q, stream)
        ws = _room(workspace, linear_attn_fwd_workspace_size(T, S, Hk, Hv, K, V, dt), q, stream)
        _check(lib().varlen_linear_attn_fwd(
            *args, float(K ** -0.5 if scale is None else scale), _ptr(cu_seqlens, "cu_seqlens", torch.int32), S, T, Hk,
            Hv, K, V, dt, op, _shaped(initial_states, "initial_states", (S, Hv, K, V)),
            _shaped(final_states, "final_states", (S, Hv, K, V)), _ptr(ws, "workspace"),
            ws.numel() * ws.element_size(), _stream_of(q, stream)), "varlen_linear_attn_fwd")
    return (out, final_states) if want_final else out


def varlen_linear_attn_bwd(q, k, v, g, dout, cu_seqlens, scale=None, grads=None, workspace=None, stream=None,
                           initial_states=None, d_final_states=None, d_initial_states=None, dg=True):
    """Returns dict dq, dk, dv, dg, d_initial_states.  The inputs,
    initial_states and scale are the forward call's.  dg: False for decays
    that are not trained (None is returned for it then).  d_final_states:
    (S, Hv, K, V) f32, the gradient reaching the final states;
    d_initial_states: None / False, True or a tensor to fill.  grads: tensors
    to fill, by name."""
    args, (T, Hk, Hv, K, V) = _linear_args(q, k, v, g)
    S, dt = _num_seqs(cu_seqlens), _dt(q)
    r = dict(grads or {})
    shapes = {"dq": ((T, Hk, K), q.dtype), "dk": ((T, Hk, K), q.dtype), "dv": ((T, Hv, V), q.dtype),
              "dg": (tuple(g.shape), torch.float32)}
    _together(q, k, v, g, dout, cu_seqlens, workspace, initial_states, d_final_states, d_initial_states, *r.values())
    with _device_of(q):
        for n, (shape, d) in shapes.items():
            if n not in r:
                r[n] = _new(shape, d, q, stream) if n != "dg" or dg else None
        r["d_initial_states"] = _asked(d_initial_states, (S, Hv, K, V), q, stream)
        ws = _room(workspace, linear_attn_bwd_workspace_size(T, S, Hk, Hv, K, V, dt), q, stream)
        _check(lib().varlen_linear_attn_bwd(
            *args, _shaped(dout, "dout", (T, Hv, V), q.dtype), float(K ** -0.5 if scale is None else scale),
            _ptr(cu_seqlens, "cu_seqlens", torch.int32), S, T, Hk, Hv, K, V, dt,
            _shaped(initial_states, "initial_states", (S, Hv, K, V)),
            _shaped(d_final_states, "d_final_states", (S, Hv, K, V)),
            _shaped(r["d_initial_states"], "d_initial_states", (S, Hv, K, V)),
            *(_shaped(r[n], n, shape, d) for n, (shape, d) in shapes.items()),
            _ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream_of(q, stream)), "varlen_linear_attn_bwd")
    return r


def varlen_linear_attn_step(q, k, v, g, states, state_indices=None, scale=None, out=None, status=None, stream=None):
    """Returns out (B, Hv, V): one token of each of B sequences, q, k (B, Hk, K),
    v (B, Hv, V), g (B, Hv) or (Hv,), against states (slots, Hv, K, V) f32,
    which are updated in place.  state_indices: int32 (B) slots, all
    different, negative for a padded entry (None: entry b uses slot b).
    status: optional int32 tensor for indices outside the pool."""
    args, (B, Hk, Hv, K, V) = _linear_args(q, k, v, g)
    if _cuda(states, "states").dim() != 4:
        raise ValueError(f"states must be (slots, {Hv}, {K}, {V}), got {tuple(states.shape)}")
    slots = states.shape[0]
    _together(q, k, v, g, states, state_indices, out, status)
    with _device_of(q):
        out, op = _result(out, "out", v, stream)
        _check(lib().varlen_linear_attn_step(
            *args, float(K ** -0.5 if scale is None else scale), _shaped(states, "states", (slots, Hv, K, V)),
            _shaped(state_indices, "state_indices", (B,), torch.int32), slots, B, Hk, Hv, K, V, _dt(q), op,
            _ptr(status, "status", torch.int32), _stream_of(q, stream)), "varlen_linear_attn_step")
    return out


# ------------------------------------------------------------------ layer norm
def _rows(t, name):
    """(pointer, row stride) of a (T, D) CUDA tensor whose rows may be any
    distance apart."""
    if _cuda(t, name).dim() != 2:
        raise ValueError(f"{name} must be (tokens, channels), got {tuple(t.shape)}")
    T, D = t.shape
    if D > 1 and t.stride(1) != 1 and t.numel():
        raise ValueError(f"{name}: the channels of a token must be contiguous")
    return t.data_ptr() or None, (t.stride(0) if T > 1 else D)


def varlen_layer_norm_fwd(x, weight=None, bias=None, groups=1, eps=1e-5, residual=None, out=None, sum_out=None,
                          stream=None):
    """Returns out, or (out, sum) with a residual: the rows of x (T, D), or of
    sum = residual + x, with mean 0 and variance 1, scaled by weight and moved
    by bias (D) f32, over all D channels or each of `groups` groups of them.
    x may be slices of wider rows; residual and sum (T, D) are float32
    whatever x is.  out, sum_out: tensors to fill (sum_out may be residual)."""
    xp, sx = _rows(x, "x")
    T, D = x.shape
    if residual is None and sum_out is not None:
        raise ValueError("sum_out needs a residual")
    _together(x, weight, bias, residual, out, sum_out)
    with _device_of(x):
        out, op = _result(out, "out", x, stream)
        rp = _shaped(residual, "residual", (T, D))
        if residual is not None and sum_out is None:
            sum_out = _new((T, D), torch.float32, x, stream)
        _check(lib().varlen_layer_norm_fwd(
            xp, sx, rp, _shaped(weight, "weight", (D,)), _shaped(bias, "bias", (D,)), T, D, int(groups), float(eps),
            _dt(x), op, _shaped(sum_out, "sum_out", (T, D)), _stream_of(x, stream)), "varlen_layer_norm_fwd")
    return out if residual is None else (out, sum_out)


def varlen_layer_norm_bwd(x, weight, bias, dout, groups=1, eps=1e-5, residual=False, dsum=None, grads=None,
                          workspace=None, stream=None):
    """Returns dict dx and, where the forward call had them, dweight, dbias and
    dresidual (else None).  x: what was normalised: the forward call's x, or,
    with residual=True, its sum, float32; dout (T, D) has dx's type.  dsum:
    (T, D) f32, the gradient that reaches the sum from elsewhere, or None.
    grads: tensors to fill, by name."""
    xp, sx = _rows(x, "x")
    T, D = x.shape
    dt = _dt(_cuda(dout, "dout"))
    want = torch.float32 if residual else dout.dtype
    if x.dtype is not want:
        raise TypeError(f"x must be {want}, got {x.dtype}")
    if dsum is not None and not residual:
        raise ValueError("dsum needs residual=True")
    g = dict(grads or {})
    make = {"dx": ((T, D), dout.dtype), "dresidual": ((T, D), torch.float32), "dweight": ((D,), torch.float32),
            "dbias": ((D,), torch.float32)}
    _together(x, weight, bias, dout, dsum, workspace, *g.values())
    _shaped(bias, "bias", (D,))  # the call needs none of its values
    with _device_of(x):
        for n, wanted in (("dx", True), ("dresidual", residual), ("dweight", weight is not None),
                          ("dbias", bias is not None)):
            if n not in g:
                g[n] = _new(*make[n], x, stream) if wanted else None
        ws = _room(workspace, lib().varlen_layer_norm_bwd_workspace_size(T, D, int(groups)), x, stream)
        _check(lib().varlen_layer_norm_bwd(
            xp, sx, int(bool(residual)), _shaped(weight, "weight", (D,)), _shaped(dout, "dout", (T, D), dout.dtype),
            _shaped(dsum, "dsum", (T, D)), T, D, int(groups), float(eps), dt,
            *(_shaped(g[n], n, *make[n]) for n in make), _ptr(ws, "workspace"), ws.numel() * ws.element_size(),
            _stream_of(x, stream)), "varlen_layer_norm_bwd")
    return g


# ------------------------------------------------------------------ packing (host)
PACK_METHODS = {"sequential": 0, "local_greedy": 1}


def pack_sequences(lengths, pack_size, method="local_greedy", window=1000):
    """Packs sequences of the given lengths into packs of at most pack_size
    tokens (host work, no GPU).  Returns (packs, padding_rate): packs is a
    list of int32 arrays of sequence indices, in pack order."""
    import numpy as np
    L = np.ascontiguousarray(lengths, dtype=np.int32)
    n = int(L.size)
    order = np.empty(max(n, 1), dtype=np.int32)
    offs = np.empty(n + 1, dtype=np.int32)
    npk, pad = ctypes.c_int32(0), ctypes.c_double(0.0)
    _check(lib().varlen_pack_sequences(L.ctypes.data if n else None, n, int(pack_size), PACK_METHODS[method],
                                       int(window), order.ctypes.data, offs.ctypes.data, ctypes.byref(npk),
                                       ctypes.byref(pad)), "varlen_pack_sequences")
    return [order[offs[p]:offs[p + 1]].copy() for p in range(npk.value)], pad.value
