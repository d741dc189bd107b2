"""Gated delta rule, the norm of queries and keys with their rotation, and the layer of both: the binding of
the third part of include/kata.h.  Like the rest of the package it marshals torch tensors into the C ABI
and enqueues the work on the current stream of the tensors' device.

    q, k = fwd_qk_norm(q, k, l2=True)                     # unit rows; bwd_qk_norm: its gradients
    o = fwd_delta(q, k, v, beta, log_decay)               # chunked form, batch or packed
    dq, dk, dv, dbeta, dlog_decay, dstate = bwd_delta(q, k, v, beta, dO, log_decay)
    o = decode_delta(q, k, v, beta, state, log_decay)     # recurrent form, state in place
    o = parallel_delta_attn(q, k, v, beta, log_decay)     # differentiable

"""

import ctypes
import struct

import torch
from torch.autograd.function import once_differentiable

from . import layer as _l
from .layer import _bytes, _dtype, _empty, _out_like, _ptr, _rows_ok, _run, _state, _workspace, _workspace_size, _written

_I32, _I64, _F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class _DeltaProblem(ctypes.Structure):
    _fields_ = [("n_seq", _I32), ("H", _I32), ("Hk", _I32), ("T", _I32), ("dk", _I32), ("dv", _I32),
                ("packed", _I32), ("zero_tail", _I32), ("dtype", _I32), ("scale", _F32),
                ("sq", _I64 * 3), ("sk", _I64 * 3), ("sv", _I64 * 3), ("so", _I64 * 3), ("sdo", _I64 * 3),
                ("sbeta", _I64 * 3), ("sdecay", _I64 * 3)]


_DELTA = struct.Struct("9if21q")
assert _DELTA.size == ctypes.sizeof(_DeltaProblem)


def _signatures():
    VP, SZ = ctypes.c_void_p, ctypes.c_size_t   # a problem is passed by its address
    return {
        "kata_fwd_delta_workspace_size": (SZ, [VP]),
        "kata_fwd_delta": (_I32, [VP] * 11 + [SZ, VP]),
        "kata_bwd_delta_workspace_size": (SZ, [VP]),
        "kata_bwd_delta": (_I32, [VP] * 17 + [SZ, VP]),
        "kata_decode_delta": (_I32, [VP] * 9),
    }


# ---- gated delta rule ----------------------------------------------------------------------------

def _delta_problem(q, k, v, beta, log_decay, scale, cu_seqlens, o=None, dO=None, zero_tail=0):
    """The packed kata_delta_problem of a call, its arguments checked."""
    device, dtype, shape = q.device, q.dtype, q.shape
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    if len(shape) != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be 4-D (B, T, H, D)")
    B, T, Hk, dk = shape
    H, dv = v.shape[2:]
    if k.shape != shape or v.shape != (B, T, H, dv) or k.dtype != dtype or v.dtype != dtype:
        raise ValueError("q, k, v must share (B, T) and dtype; q and k share heads and dk")
    if Hk == 0 or H % Hk:
        raise ValueError("v's heads must be a multiple of q's and k's")
    if beta.shape != (B, T, H) or beta.dtype != dtype:
        raise ValueError("beta must have the inputs' dtype and shape (B, T, H)")
    if k.device != device or v.device != device or beta.device != device or (o is not None and o.device != device):
        raise ValueError(f"k, v, beta, log_decay and out must be on {device}")
    sl = (0, 0, 0)
    if log_decay is not None:
        if log_decay.shape != (B, T, H) or log_decay.dtype != torch.float32 or log_decay.device != device:
            raise ValueError(f"log_decay must be fp32 of shape (B, T, H) on {device}")
        sl = log_decay.stride()
    n, packed = B, 0
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or cu_seqlens.dtype != torch.int32 \
                or not cu_seqlens.is_contiguous() or cu_seqlens.device != device:
            raise ValueError(f"cu_seqlens must be a contiguous int32 tensor of n + 1 >= 2 offsets on {device}")
        if B != 1:
            raise ValueError("packed sequences lie in one batch row: B must be 1")
        n, packed = cu_seqlens.numel() - 1, 1
    sq, sk, sv = q.stride(), k.stride(), v.stride()
    so = (T * H * dv, H * dv, dv, 1) if o is None else o.stride()
    sdo = so
    if dO is not None:
        sdo = dO.stride()
        if dO.device != device:
            raise ValueError(f"dO must be on {device}")
    if not sq[3] == sk[3] == sv[3] == so[3] == sdo[3] == 1:
        for name, x in (("q", q), ("k", k), ("v", v), ("out", o), ("dO", dO)):
            if x is not None:
                _rows_ok(x, name)
    return _DELTA.pack(n, H, Hk, T, dk, dv, packed, zero_tail, _dtype(dtype), scale, *sq[:3], *sk[:3], *sv[:3],
                       *so[:3], *sdo[:3], *beta.stride(), *sl)


def delta_state_shape(q, v, cu_seqlens=None):
    """Shape of the states of (B, T, Hk, dk) queries and (B, T, H, dv) values: (n, H, dk, dv) fp32 for n
    sequences."""
    n = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    return (n, v.shape[2], q.shape[3], v.shape[3])


def fwd_delta(q, k, v, beta, log_decay=None, scale=1.0, initial_state=None, return_state=False,
              cu_seqlens=None, out=None, workspace=None):
    """o_t = scale S_t^T q_t with S_t = g_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T and g_t =
    exp(log_decay_t), in chunks (MFMA).

    q, k (B, T, Hk, dk), v (B, T, H, dv), H a multiple of Hk (value head h uses head h // (H / Hk)), bf16 or
    fp32, widths up to 128 with rows of whole 16 bytes, any (b, t, h) strides that keep rows apart, or zero
    (broadcast axes).  beta (B, T, H) in the inputs' dtype; log_decay fp32 (B, T, H), or None (no decay).  Keys of
    unit length and beta in [0, 2] keep the state bounded.  o has v's shape and dtype.
    cu_seqlens: int32 (n + 1,) offsets of n sequences packed into B = 1; rows of no sequence are zero in a
    new output and left as they are in `out`, which must not overlap an input.
    initial_state, and the final state with return_state: fp32 (n, H, dk, dv).  Sums and states are fp32; bf16
    operands that come out of them are kept in two terms (2^-18).
    workspace: uint8, delta_workspace_size() bytes (allocated here otherwise)."""
    o = _out_like(v, out)
    pr = _delta_problem(q, k, v, beta, log_decay, scale, cu_seqlens, o=o, zero_tail=1 if out is None else 0)
    shape, device = delta_state_shape(q, v, cu_seqlens), q.device
    _state(initial_state, shape, device, "initial_state")
    final = torch.empty(shape, dtype=torch.float32, device=device) if return_state else None
    if q.shape[0] * q.shape[1] == 0:
        if final is not None:
            final.copy_(initial_state) if initial_state is not None else final.zero_()
    elif v.shape[2]:
        ws = _workspace(_workspace_size("kata_fwd_delta_workspace_size", pr), workspace, device)
        _run("kata_fwd_delta", device, pr, q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(),
             _ptr(log_decay), _ptr(cu_seqlens), _ptr(initial_state), o.data_ptr(), _ptr(final), _ptr(ws), _bytes(ws))
    if out is not None:
        _written(out)
    return (o, final) if return_state else o


def delta_workspace_size(q, k, v, beta, log_decay=None, cu_seqlens=None, backward=False):
    """Bytes of workspace fwd_delta (or bwd_delta) needs."""
    return _workspace_size(f"kata_{'bwd' if backward else 'fwd'}_delta_workspace_size",
                           _delta_problem(q, k, v, beta, log_decay, 1.0, cu_seqlens))


def bwd_delta(q, k, v, beta, dO, log_decay=None, scale=1.0, initial_state=None, dfinal_state=None,
              cu_seqlens=None, workspace=None):
    """Gradients (dq, dk, dv, dbeta, dlog_decay, dinitial_state) of sum(dO * o) + sum(dfinal_state *
    final_state): the first four in the inputs' dtype (dq and dk summed over the value heads of a head), the
    others fp32 (None without a log_decay or an initial_state).  Rows of no packed sequence get zeros."""
    if dO.shape != v.shape or dO.dtype != q.dtype:
        raise ValueError("dO must match v's shape and q's dtype")
    pr = _delta_problem(q, k, v, beta, log_decay, scale, cu_seqlens, dO=dO, zero_tail=1)
    shape, device = delta_state_shape(q, v, cu_seqlens), q.device
    _state(initial_state, shape, device, "initial_state")
    _state(dfinal_state, shape, device, "dfinal_state")
    dq, dk, dv, db = _empty(q), _empty(k), _empty(v), _empty(beta)
    dl = None if log_decay is None else _empty(log_decay)
    dinit = torch.empty(shape, dtype=torch.float32, device=device) if initial_state is not None else None
    if q.shape[0] * q.shape[1] == 0:
        if dinit is not None:
            dinit.copy_(dfinal_state) if dfinal_state is not None else dinit.zero_()
    elif v.shape[2]:
        ws = _workspace(_workspace_size("kata_bwd_delta_workspace_size", pr), workspace, device)
        _run("kata_bwd_delta", device, pr, q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(),
             _ptr(log_decay), dO.data_ptr(), _ptr(cu_seqlens), _ptr(initial_state), _ptr(dfinal_state),
             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), db.data_ptr(), _ptr(dl), _ptr(dinit), _ptr(ws), _bytes(ws))
    else:
        dq.zero_(), dk.zero_()
    return dq, dk, dv, db, dl, dinit


def decode_delta(q, k, v, beta, state, log_decay=None, scale=1.0, out=None):
    """Advances `state` (fp32 (B, H, dk, dv), in place) over the T tokens of q, k, v one at a time and
    returns o; T = 1 is one decode step.  All arithmetic is fp32."""
    o = _out_like(v, out)
    pr = _delta_problem(q, k, v, beta, log_decay, scale, None, o=o)
    if state is None:
        raise ValueError("decode_delta needs a state")
    _state(state, delta_state_shape(q, v), q.device, "state")
    if v.numel():
        _run("kata_decode_delta", q.device, pr, q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(),
             _ptr(log_decay), state.data_ptr(), o.data_ptr())
    _written(state if out is None else (state, out))
    return o
