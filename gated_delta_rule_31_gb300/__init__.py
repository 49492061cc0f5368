"""GB300 (sm_103a) gated delta rule: thin Python binding of the C ABI in ``include/gdr.h``.

Every step of the computation runs in ``libgdr.so``'s CUDA kernels; this module only
checks tensors, allocates outputs and workspace with torch, and passes raw device
pointers and the current CUDA stream through ctypes. There is no CPU fallback: if the
library is missing or a tensor is not on a CUDA device, the calls raise.

Operation (Gated DeltaNet recurrence, per batch and value head, key head hv // (Hv/Hk)):
    k^ = k (|k|^2 + 1e-6)^-1/2,  q^ likewise      (when use_qk_l2norm)
    S_t = S_{t-1} diag(exp g_t) (I - beta_t k^ k^T) + beta_t v_t k^T,   o_t = scale S_t q^
Layouts: q,k [B,T,Hk,Dk]; v,o [B,T,Hv,Dv]; g [B,T,Hv] or [B,T,Hv,Dk] fp32; beta [B,T,Hv]
fp32; states [B,Hv,Dv,Dk] fp32.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from ._build import LIB as _LIB_PATH
from ._build import build

__all__ = ["build", "fwd_chunked", "bwd_chunked", "fwd_sequential", "bwd_sequential", "decode_step", "GdrError",
           "fwd_workspace_bytes", "bwd_workspace_bytes", "lib", "Problem", "workspace_status", "selftest_wait_expiry", "trace",
           "LinearProblem", "NormProblem", "linear_fwd", "linear_bwd", "linear_decode_step", "group_norm_fwd",
           "group_norm_bwd"]

GDR_F32, GDR_BF16 = 0, 1
GDR_GATE_SCALAR, GDR_GATE_CHANNEL = 0, 1
GDR_ERR_INVALID_ARG, GDR_ERR_UNSUPPORTED = 1, 2
_ACTIVATIONS = {"none": 0, "silu": 1, "sigmoid": 2}


class Problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hk", ctypes.c_int), ("Hv", ctypes.c_int),
                ("Dk", ctypes.c_int), ("Dv", ctypes.c_int), ("dtype", ctypes.c_int), ("gate", ctypes.c_int),
                ("scale", ctypes.c_float), ("use_qk_l2norm", ctypes.c_int)]


class LinearProblem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hk", ctypes.c_int), ("Hv", ctypes.c_int),
                ("Dk", ctypes.c_int), ("Dv", ctypes.c_int), ("dtype", ctypes.c_int), ("scale", ctypes.c_float)]


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("groups", ctypes.c_int), ("D", ctypes.c_int), ("dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("center", ctypes.c_int), ("eps", ctypes.c_float)]


class GdrError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(msg)
        self.code = code


_lib = None


def lib():
    """The loaded libgdr.so (ctypes handle). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it first (gated_delta_rule_31_gb300.build())")
        L = ctypes.CDLL(_LIB_PATH)
        P, PP, sz, st = ctypes.c_void_p, ctypes.POINTER(Problem), ctypes.c_size_t, ctypes.c_void_p
        L.gdr_status_string.argtypes = [ctypes.c_int]
        L.gdr_status_string.restype = ctypes.c_char_p
        L.gdr_fwd_chunked_workspace.argtypes = [PP]
        L.gdr_fwd_chunked_workspace.restype = sz
        L.gdr_bwd_chunked_workspace.argtypes = [PP]
        L.gdr_bwd_chunked_workspace.restype = sz
        L.gdr_fwd_chunked.argtypes = [PP] + [P] * 8 + [P, sz, st]
        L.gdr_fwd_chunked.restype = ctypes.c_int
        L.gdr_fwd_sequential.argtypes = [PP] + [P] * 8 + [st]
        L.gdr_fwd_sequential.restype = ctypes.c_int
        L.gdr_bwd_chunked.argtypes = [PP] + [P] * 14 + [P, sz, st]
        L.gdr_bwd_sequential_workspace.argtypes = [PP]
        L.gdr_bwd_sequential_workspace.restype = sz
        L.gdr_bwd_sequential.argtypes = [PP] + [P] * 14 + [P, sz, st]
        L.gdr_bwd_sequential.restype = ctypes.c_int
        L.gdr_bwd_chunked.restype = ctypes.c_int
        L.gdr_decode_step.argtypes = [PP] + [P] * 7 + [st]
        L.gdr_decode_step.restype = ctypes.c_int
        L.gdr_chunk_states_bytes.argtypes = [PP]
        L.gdr_chunk_states_bytes.restype = sz
        L.gdr_bwd_chunked_states_workspace.argtypes = [PP]
        L.gdr_bwd_chunked_states_workspace.restype = sz
        L.gdr_fwd_chunked_states.argtypes = [PP] + [P] * 8 + [P, sz, P, sz, st]
        L.gdr_fwd_chunked_states.restype = ctypes.c_int
        L.gdr_bwd_chunked_states.argtypes = [PP] + [P] * 5 + [P, sz] + [P] * 8 + [P, sz, st]
        L.gdr_bwd_chunked_states.restype = ctypes.c_int
        for name in ("gdr_chunk_saved_bytes", "gdr_fwd_chunked_saved_workspace", "gdr_bwd_chunked_saved_workspace"):
            getattr(L, name).argtypes = [PP]
            getattr(L, name).restype = sz
        L.gdr_fwd_chunked_saved.argtypes = [PP] + [P] * 8 + [P, sz, P, sz, st]
        L.gdr_fwd_chunked_saved.restype = ctypes.c_int
        L.gdr_bwd_chunked_saved.argtypes = [PP] + [P] * 5 + [P, sz] + [P] * 8 + [P, sz, st]
        L.gdr_bwd_chunked_saved.restype = ctypes.c_int
        L.gdr_workspace_status.argtypes = [P, sz, st]
        L.gdr_workspace_status.restype = ctypes.c_int
        L.gdr_selftest_wait_expiry.argtypes = [P, sz, st]
        L.gdr_selftest_wait_expiry.restype = ctypes.c_int
        L.gdr_trace_enable.argtypes = [ctypes.c_int]
        L.gdr_trace_enable.restype = ctypes.c_int
        L.gdr_trace_collect.argtypes = [ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float),
                                        ctypes.c_int]
        L.gdr_trace_collect.restype = ctypes.c_int
        PL, PN = ctypes.POINTER(LinearProblem), ctypes.POINTER(NormProblem)
        for name, at in (("gdr_linear_fwd_workspace", PL), ("gdr_linear_bwd_workspace", PL),
                         ("gdr_linear_states_bytes", PL), ("gdr_linear_bwd_states_workspace", PL),
                         ("gdr_group_norm_bwd_workspace", PN)):
            getattr(L, name).argtypes = [at]
            getattr(L, name).restype = sz
        L.gdr_linear_fwd.argtypes = [PL] + [P] * 8 + [P, sz, st]
        L.gdr_linear_bwd.argtypes = [PL] + [P] * 12 + [P, sz, st]
        L.gdr_linear_fwd_states.argtypes = [PL] + [P] * 8 + [P, sz, P, sz, st]
        L.gdr_linear_bwd_states.argtypes = [PL] + [P] * 6 + [P, sz] + [P] * 6 + [P, sz, st]
        L.gdr_linear_decode_step.argtypes = [PL] + [P] * 6 + [st]
        L.gdr_group_norm_fwd.argtypes = [PN] + [P] * 5 + [st]
        L.gdr_group_norm_bwd.argtypes = [PN] + [P] * 9 + [P, sz, st]
        for name in ("gdr_linear_fwd", "gdr_linear_bwd", "gdr_linear_fwd_states", "gdr_linear_bwd_states",
                     "gdr_linear_decode_step", "gdr_group_norm_fwd", "gdr_group_norm_bwd"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(code: int):
    if code != 0:
        raise GdrError(code, lib().gdr_status_string(code).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _written(*tensors):
    """Tells autograd that a call wrote these tensors of the caller's: a graph that saved one refuses its backward."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _need(t, name, dtype=None, device=None, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _problem(q, v, g, scale, use_qk_l2norm, T=None):
    if q.dim() == 4:
        B, T_, Hk, Dk = q.shape
    else:  # decode: [B, Hk, Dk]
        B, Hk, Dk = q.shape
        T_ = 1
    Hv, Dv = v.shape[-2], v.shape[-1]
    channel = g.dim() == (4 if q.dim() == 4 else 3)
    dtype = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16}.get(q.dtype)
    if dtype is None:
        raise ValueError(f"q/k/v dtype must be float32 or bfloat16, got {q.dtype}")
    if scale is None:
        scale = Dk ** -0.5
    return Problem(B, T_ if T is None else T, Hk, Hv, Dk, Dv, dtype,
                   GDR_GATE_CHANNEL if channel else GDR_GATE_SCALAR, float(scale), int(bool(use_qk_l2norm)))


def _check_inputs(q, k, v, g, beta, h0=None):
    dev = q.device
    _need(q, "q", device=dev)
    _need(k, "k", dtype=q.dtype, device=dev, shape=q.shape)
    _need(v, "v", dtype=q.dtype, device=dev)
    _need(g, "g", dtype=torch.float32, device=dev)
    _need(beta, "beta", dtype=torch.float32, device=dev)
    lead = tuple(q.shape[:-2])
    Hv, Dv, Dk = v.shape[-2], v.shape[-1], q.shape[-1]
    if tuple(v.shape[:-2]) != lead:
        raise ValueError("v leading dims must match q")
    if tuple(beta.shape) != lead + (Hv,):
        raise ValueError(f"beta must be {lead + (Hv,)}")
    if tuple(g.shape) not in (lead + (Hv,), lead + (Hv, Dk)):
        raise ValueError(f"g must be {lead + (Hv,)} or {lead + (Hv, Dk)}")
    if h0 is not None:
        _need(h0, "h0", dtype=torch.float32, device=dev, shape=(q.shape[0], Hv, Dv, Dk))


def fwd_workspace_bytes(p: Problem) -> int:
    return int(lib().gdr_fwd_chunked_workspace(ctypes.byref(p)))


def bwd_workspace_bytes(p: Problem) -> int:
    return int(lib().gdr_bwd_chunked_workspace(ctypes.byref(p)))


def _workspace(query, p, device, workspace, missing=GDR_ERR_UNSUPPORTED):
    """(workspace, bytes) for the call whose size query is `query`: the caller's tensor after
    checking it, else a new uint8 buffer. A zero size means the call does not take this problem
    and raises as the status `missing` would."""
    nbytes = int(query(ctypes.byref(p)))
    if nbytes == 0:
        _check(missing)
    if workspace is not None:
        _need(workspace, "workspace", device=device)
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace too small: {workspace.numel() * workspace.element_size()} < {nbytes} bytes")
        return workspace, nbytes
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device), nbytes


def fwd_sequential(q, k, v, g, beta, h0=None, scale=None, use_qk_l2norm=True, output_final_state=True):
    """Token-by-token forward (gdr_fwd_sequential). Returns (o, ht or None)."""
    _check_inputs(q, k, v, g, beta, h0)
    p = _problem(q, v, g, scale, use_qk_l2norm)
    o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    ht = torch.empty((p.B, p.Hv, p.Dv, p.Dk), dtype=torch.float32, device=v.device) if output_final_state else None
    _check(lib().gdr_fwd_sequential(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                    _ptr(o), _ptr(ht), _stream(q.device)))
    return o, ht


def fwd_chunked(q, k, v, g, beta, h0=None, scale=None, use_qk_l2norm=True, output_final_state=True,
                workspace=None, save_states=False, save_all=False):
    """Chunked prefill forward (gdr_fwd_chunked: bf16 on the tensor cores, fp32 on the CUDA-core
    fp32 kernels). Returns (o, ht or None),
    or (o, ht, states) with save_states=True (gdr_fwd_chunked_states: the chunk-start states
    kept for bwd_chunked(..., states=states)), or (o, ht, saved) with save_all=True
    (gdr_fwd_chunked_saved: states and chunk operators kept for bwd_chunked(..., saved=saved))."""
    _check_inputs(q, k, v, g, beta, h0)
    p = _problem(q, v, g, scale, use_qk_l2norm)
    o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    ht = torch.empty((p.B, p.Hv, p.Dv, p.Dk), dtype=torch.float32, device=v.device) if output_final_state else None
    if save_all:
        L = lib()
        ws, nbytes = _workspace(L.gdr_fwd_chunked_saved_workspace, p, q.device, workspace)
        sb = int(L.gdr_chunk_saved_bytes(ctypes.byref(p)))
        saved = torch.empty(max(sb, 256), dtype=torch.uint8, device=q.device)
        _check(L.gdr_fwd_chunked_saved(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                       _ptr(o), _ptr(ht), _ptr(saved), ctypes.c_size_t(sb), _ptr(ws),
                                       ctypes.c_size_t(nbytes), _stream(q.device)))
        return o, ht, saved
    ws, nbytes = _workspace(lib().gdr_fwd_chunked_workspace, p, q.device, workspace)
    if not save_states:
        _check(lib().gdr_fwd_chunked(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                     _ptr(o), _ptr(ht), _ptr(ws), ctypes.c_size_t(nbytes), _stream(q.device)))
        return o, ht
    sb = int(lib().gdr_chunk_states_bytes(ctypes.byref(p)))
    states = torch.empty(max(sb, 256), dtype=torch.uint8, device=q.device)
    _check(lib().gdr_fwd_chunked_states(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                        _ptr(o), _ptr(ht), _ptr(states), ctypes.c_size_t(sb), _ptr(ws),
                                        ctypes.c_size_t(nbytes), _stream(q.device)))
    return o, ht, states


def bwd_chunked(q, k, v, g, beta, h0, do, dht=None, scale=None, use_qk_l2norm=True, workspace=None,
                states=None, saved=None):
    """Chunked backward (gdr_bwd_chunked) of <do,o> + <dht,ht>. Returns a dict of fp32
    gradients dq, dk, dv, dg, dbeta, dh0. With `states` from fwd_chunked(save_states=True)
    on the same inputs, gdr_bwd_chunked_states reads them instead of re-running the
    forward scan; with `saved` from fwd_chunked(save_all=True), gdr_bwd_chunked_saved runs
    neither prep nor the forward scan (h0 is unused in both cases)."""
    _check_inputs(q, k, v, g, beta, h0)
    _need(do, "do", dtype=v.dtype, device=v.device, shape=v.shape)
    p = _problem(q, v, g, scale, use_qk_l2norm)
    if dht is not None:
        _need(dht, "dht", dtype=torch.float32, device=v.device, shape=(p.B, p.Hv, p.Dv, p.Dk))
    f32 = dict(dtype=torch.float32, device=v.device)
    out = dict(dq=torch.empty(q.shape, **f32), dk=torch.empty(k.shape, **f32), dv=torch.empty(v.shape, **f32),
               dg=torch.empty(g.shape, **f32), dbeta=torch.empty(beta.shape, **f32),
               dh0=torch.empty((p.B, p.Hv, p.Dv, p.Dk), **f32))
    if saved is not None:
        _need(saved, "saved", dtype=torch.uint8, device=q.device)
        L = lib()
        ws, nbytes = _workspace(L.gdr_bwd_chunked_saved_workspace, p, q.device, workspace)
        _check(L.gdr_bwd_chunked_saved(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                       _ptr(saved), ctypes.c_size_t(saved.numel()), _ptr(do), _ptr(dht),
                                       _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                                       _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(ws), ctypes.c_size_t(nbytes),
                                       _stream(q.device)))
        return out
    if states is None:
        ws, nbytes = _workspace(lib().gdr_bwd_chunked_workspace, p, q.device, workspace)
        _check(lib().gdr_bwd_chunked(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                     _ptr(do), _ptr(dht), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                     _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(ws),
                                     ctypes.c_size_t(nbytes), _stream(q.device)))
        return out
    _need(states, "states", dtype=torch.uint8, device=q.device)
    ws, nbytes = _workspace(lib().gdr_bwd_chunked_states_workspace, p, q.device, workspace)
    _check(lib().gdr_bwd_chunked_states(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                        _ptr(states), ctypes.c_size_t(states.numel()), _ptr(do), _ptr(dht),
                                        _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                                        _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(ws), ctypes.c_size_t(nbytes),
                                        _stream(q.device)))
    return out


def bwd_sequential(q, k, v, g, beta, h0, do, dht=None, scale=None, use_qk_l2norm=True, workspace=None):
    """Sequential VJP (gdr_bwd_sequential) of <do,o> + <dht,ht>: every dtype, gate and head
    size. Returns a dict of fp32 gradients dq, dk, dv, dg, dbeta, dh0 (dg has g's shape)."""
    _check_inputs(q, k, v, g, beta, h0)
    _need(do, "do", dtype=v.dtype, device=v.device, shape=v.shape)
    p = _problem(q, v, g, scale, use_qk_l2norm)
    if dht is not None:
        _need(dht, "dht", dtype=torch.float32, device=v.device, shape=(p.B, p.Hv, p.Dv, p.Dk))
    f32 = dict(dtype=torch.float32, device=v.device)
    out = dict(dq=torch.empty(q.shape, **f32), dk=torch.empty(k.shape, **f32), dv=torch.empty(v.shape, **f32),
               dg=torch.empty(g.shape, **f32), dbeta=torch.empty(beta.shape, **f32),
               dh0=torch.empty((p.B, p.Hv, p.Dv, p.Dk), **f32))
    ws, nbytes = _workspace(lib().gdr_bwd_sequential_workspace, p, q.device, workspace, missing=GDR_ERR_INVALID_ARG)
    _check(lib().gdr_bwd_sequential(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                    _ptr(do), _ptr(dht), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                                    _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(ws),
                                    ctypes.c_size_t(nbytes), _stream(q.device)))
    return out


def decode_step(q, k, v, g, beta, state, scale=None, use_qk_l2norm=True, out=None):
    """One decode step (gdr_decode_step): q,k [B,Hk,Dk]; v [B,Hv,Dv]; g [B,Hv] or [B,Hv,Dk];
    beta [B,Hv]; state [B,Hv,Dv,Dk] fp32 updated in place. Returns o [B,Hv,Dv]."""
    _check_inputs(q, k, v, g, beta)
    p = _problem(q, v, g, scale, use_qk_l2norm)
    _need(state, "state", dtype=torch.float32, device=q.device, shape=(p.B, p.Hv, p.Dv, p.Dk))
    if out is not None:
        _need(out, "out", dtype=v.dtype, device=v.device, shape=v.shape)
    o = out if out is not None else torch.empty(v.shape, dtype=v.dtype, device=v.device)
    _check(lib().gdr_decode_step(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                                 _ptr(o), _stream(q.device)))
    _written(state, out)
    return o


# The calls below are short enough for the host's part to matter: tensors are compared with what they
# have to be in one expression each (_need only words the refusal), pointers go as plain integers, and the
# problem with its buffer sizes is built once for each set of sizes.
_DTYPES = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16}


def _is(t, name, dtype, device, shape):
    if not (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        _need(t, name, dtype=dtype, device=device, shape=shape)


def _at(t):
    return None if t is None else t.data_ptr()


def _raw_stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


@functools.lru_cache(maxsize=1024)
def _linear_spec(B, T, Hk, Hv, Dk, Dv, dtype, scale):
    """(by-reference problem, bytes: forward workspace, kept states, backward workspace without and with them)."""
    p, L = LinearProblem(B, T, Hk, Hv, Dk, Dv, dtype, scale), lib()
    at = ctypes.byref(p)
    return at, tuple(int(f(at)) for f in (L.gdr_linear_fwd_workspace, L.gdr_linear_states_bytes,
                                          L.gdr_linear_bwd_workspace, L.gdr_linear_bwd_states_workspace))


def _linear_problem(q, k, v, g, scale, decode):
    """Checks q, k, v, g of a linear attention call: (problem, its buffer sizes, device, state shape)."""
    qs, vs, dev, dtype = q.shape, v.shape, q.device, q.dtype
    nd = 3 if decode else 4
    if not (q.is_cuda and q.is_contiguous()):
        _need(q, "q")
    if len(qs) != nd or len(vs) != nd:
        raise ValueError(f"q and v must have {nd} dimensions")
    if dtype not in _DTYPES:
        raise ValueError(f"q/k/v dtype must be float32 or bfloat16, got {dtype}")
    _is(k, "k", dtype, dev, qs)
    _is(v, "v", dtype, dev, qs[:-2] + vs[-2:])
    Hv, Dk, Dv = vs[-2], qs[-1], vs[-1]
    _is(g, "g", torch.float32, dev, (Hv,))
    at, sizes = _linear_spec(qs[0], 1 if decode else qs[1], qs[-2], Hv, Dk, Dv, _DTYPES[dtype],
                             Dk ** -0.5 if scale is None else float(scale))
    return at, sizes, dev, (qs[0], Hv, Dv, Dk)


def _linear_extras(dev, state, h0, lengths):
    if h0 is not None:
        _is(h0, "h0", torch.float32, dev, state)
    if lengths is not None:
        _is(lengths, "lengths", torch.int32, dev, state[:1])


def _scratch(nbytes, device, workspace):
    """The caller's workspace after checking it, else a new buffer: an empty one for a problem without a
    size, which the call itself refuses with the status that says why."""
    if workspace is None or nbytes == 0:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    _need(workspace, "workspace", device=device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"workspace too small: {workspace.numel() * workspace.element_size()} < {nbytes} bytes")
    return workspace


def linear_fwd(q, k, v, g, h0=None, scale=None, lengths=None, output_final_state=True, workspace=None,
               save_states=False):
    """Linear attention with a constant decay per head over T tokens (gdr_linear_fwd):
    S_t = exp(g) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t. q, k [B,T,Hk,Dk] and v [B,T,Hv,Dv] bf16
    or fp32; g [Hv] fp32 log-decay (<= 0); h0 [B,Hv,Dv,Dk] fp32 or None (zero); lengths [B] int32
    (device) or None: entry b has lengths[b] tokens, o is zero past them and ht is the state after
    the last one. scale defaults to Dk^-1/2. Returns (o, ht or None), or (o, ht, states) with
    save_states=True (gdr_linear_fwd_states: what linear_bwd(..., states=states) need not form again)."""
    at, sizes, dev, state = _linear_problem(q, k, v, g, scale, False)
    _linear_extras(dev, state, h0, lengths)
    o = torch.empty_like(v)
    ht = torch.empty(state, dtype=torch.float32, device=dev) if output_final_state else None
    ws = _scratch(sizes[0], dev, workspace)
    ins = (at, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _at(h0), _at(lengths), o.data_ptr(), _at(ht))
    if not save_states:
        _check(lib().gdr_linear_fwd(*ins, ws.data_ptr(), sizes[0], _raw_stream(dev)))
        return o, ht
    states = torch.empty(max(sizes[1], 256), dtype=torch.uint8, device=dev)
    _check(lib().gdr_linear_fwd_states(*ins, states.data_ptr(), states.numel(), ws.data_ptr(), sizes[0],
                                       _raw_stream(dev)))
    return o, ht, states


def linear_bwd(q, k, v, g, h0, do, dht=None, scale=None, lengths=None, workspace=None, states=None, need_dh0=True):
    """VJP of linear_fwd for the loss <do, o> + <dht, ht> (gdr_linear_bwd, or gdr_linear_bwd_states
    with the `states` of linear_fwd(save_states=True) on the same inputs). Returns a dict of dq,
    dk, dv in the inputs' dtype and dh0 fp32 (None with need_dh0=False); the decay is a constant and
    has no gradient."""
    at, sizes, dev, state = _linear_problem(q, k, v, g, scale, False)
    _linear_extras(dev, state, h0, lengths)
    _is(do, "do", v.dtype, dev, v.shape)
    if dht is not None:
        _is(dht, "dht", torch.float32, dev, state)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dh0 = torch.empty(state, dtype=torch.float32, device=dev) if need_dh0 else None
    need = sizes[2] if states is None else sizes[3]
    ws = _scratch(need, dev, workspace)
    ins = (at, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _at(h0), _at(lengths))
    rest = (do.data_ptr(), _at(dht), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _at(dh0), ws.data_ptr(), need,
            _raw_stream(dev))
    if states is None:
        _check(lib().gdr_linear_bwd(*ins, *rest))
    else:
        _need(states, "states", dtype=torch.uint8, device=dev)
        _check(lib().gdr_linear_bwd_states(*ins, states.data_ptr(), states.numel(), *rest))
    return dict(dq=dq, dk=dk, dv=dv, dh0=dh0)


def linear_decode_step(q, k, v, g, state, scale=None, out=None):
    """One token of linear attention (gdr_linear_decode_step): q, k [B,Hk,Dk]; v [B,Hv,Dv]; g [Hv];
    state [B,Hv,Dv,Dk] fp32 updated in place. Returns o [B,Hv,Dv]."""
    at, _, dev, shape = _linear_problem(q, k, v, g, scale, True)
    _is(state, "state", torch.float32, dev, shape)
    o = torch.empty_like(v) if out is None else out
    if out is not None:
        _is(out, "out", v.dtype, dev, v.shape)
    _check(lib().gdr_linear_decode_step(at, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), state.data_ptr(),
                                        o.data_ptr(), _raw_stream(dev)))
    _written(state, out)
    return o


@functools.lru_cache(maxsize=1024)
def _norm_spec(rows, groups, D, dtype, activation, center, eps):
    """(by-reference problem, bytes of the backward's workspace)."""
    at = ctypes.byref(NormProblem(rows, groups, D, dtype, activation, center, eps))
    return at, int(lib().gdr_group_norm_bwd_workspace(at))


def _norm_problem(x, groups, weight, bias, gate, activation, eps, center):
    """Checks the inputs of a group norm call: (problem, backward workspace bytes, device)."""
    shape, dev, dtype = x.shape, x.device, x.dtype
    if not (x.is_cuda and x.is_contiguous()):
        _need(x, "x")
    if dtype not in _DTYPES:
        raise ValueError(f"x dtype must be float32 or bfloat16, got {dtype}")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, got {activation!r}")
    C = shape[-1] if len(shape) > 0 else 0
    if groups < 1 or C < 1 or C % groups:
        raise ValueError(f"x's last dimension must be a positive multiple of groups = {groups}, got {tuple(shape)}")
    if gate is not None:
        _is(gate, "gate", dtype, dev, shape)
    if weight is not None:
        _is(weight, "weight", torch.float32, dev, shape[-1:])
    if bias is not None:
        _is(bias, "bias", torch.float32, dev, shape[-1:])
    at, nbytes = _norm_spec(x.numel() // C, groups, C // groups, _DTYPES[dtype], _ACTIVATIONS[activation],
                            int(bool(center)), float(eps))
    return at, nbytes, dev


def group_norm_fwd(x, groups, weight=None, bias=None, gate=None, activation="none", eps=1e-5, center=True, out=None):
    """Group norm over the channels of each token (gdr_group_norm_fwd): x [..., C] bf16 or fp32,
    normalised by `groups` runs of C / groups channels with statistics of that token alone, then
    n = weight h + bias and y = act(n), or n act(gate) with a gate of x's shape. weight, bias [C]
    fp32 or None; activation "none", "silu" or "sigmoid"; center=False leaves the mean in (the
    root-mean-square form). Returns y in x's dtype; `out` may be x or gate themselves."""
    at, _, dev = _norm_problem(x, groups, weight, bias, gate, activation, eps, center)
    y = torch.empty_like(x) if out is None else out
    if out is not None:
        _is(out, "out", x.dtype, dev, x.shape)
    _check(lib().gdr_group_norm_fwd(at, x.data_ptr(), _at(gate), _at(weight), _at(bias), y.data_ptr(),
                                    _raw_stream(dev)))
    _written(out)
    return y


def group_norm_bwd(x, groups, weight, bias, gate, dy, activation="none", eps=1e-5, center=True, workspace=None):
    """VJP of group_norm_fwd (gdr_group_norm_bwd). Returns a dict of dx, dgate (x's dtype; dgate None
    without a gate), dweight and dbias (fp32; None where the parameter is)."""
    at, nbytes, dev = _norm_problem(x, groups, weight, bias, gate, activation, eps, center)
    _is(dy, "dy", x.dtype, dev, x.shape)
    dx = torch.empty_like(x)
    dgate = None if gate is None else torch.empty_like(gate)
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    ws = _scratch(nbytes, dev, workspace)
    _check(lib().gdr_group_norm_bwd(at, x.data_ptr(), _at(gate), _at(weight), _at(bias), dy.data_ptr(), dx.data_ptr(),
                                    _at(dgate), _at(dweight), _at(dbias), ws.data_ptr(), nbytes, _raw_stream(dev)))
    return dict(dx=dx, dgate=dgate, dweight=dweight, dbias=dbias)


def workspace_status(ws) -> int:
    """Reads and clears the status word of a chunked or linear attention workspace (0 = ok, 5 = a wait expired)."""
    return int(lib().gdr_workspace_status(_ptr(ws), ctypes.c_size_t(ws.numel()), _stream(ws.device)))


def selftest_wait_expiry(ws) -> None:
    """gdr_selftest_wait_expiry: one CTA's bounded wait on a phase that nothing completes gives up
    after about a second and records GDR_ERR_TIMEOUT in the status word of ``ws`` (uint8, >= 256
    bytes, on the GPU); read it back with workspace_status."""
    _check(lib().gdr_selftest_wait_expiry(_ptr(ws), ctypes.c_size_t(ws.numel()), _stream(ws.device)))


class trace:
    """Context manager recording (kernel name, ms) for every library launch inside it:
    ``with gdr.trace() as t: ...`` then ``t.records``."""

    def __enter__(self):
        lib().gdr_trace_collect(None, None, 0)
        lib().gdr_trace_enable(1)
        self.records = []
        return self

    def __exit__(self, *exc):
        L = lib()
        L.gdr_trace_enable(0)
        n = L.gdr_trace_collect(None, None, 0) if exc[0] is not None else None
        if n is None:
            cap = 1 << 16
            names = (ctypes.c_char_p * cap)()
            ms = (ctypes.c_float * cap)()
            n = L.gdr_trace_collect(names, ms, cap)
            self.records = [(names[i].decode(), float(ms[i])) for i in range(min(n, cap))]
        return False
