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


class _QkNormProblem(ctypes.Structure):
    _fields_ = [("B", _I32), ("T", _I32), ("H", _I32), ("Hk", _I32), ("D", _I32), ("rot", _I32),
                ("dtype", _I32), ("w_dtype", _I32), ("interleaved", _I32), ("l2", _I32),
                ("pos64", _I32), ("n_axes", _I32), ("magnitude", _F32), ("eps", _F32),
                ("pos_a", _I64), ("pos_b", _I64), ("pos_t", _I64), ("offset", _I64),
                ("sq", _I64 * 3), ("sk", _I64 * 3), ("soq", _I64 * 3), ("sok", _I64 * 3),
                ("sdq", _I64 * 3), ("sdk", _I64 * 3)]


# The same layouts for struct.pack: a call of a few microseconds is mostly spent in its arguments.
_DELTA = struct.Struct("9if21q")
_QK_NORM = struct.Struct("12i2f22q")
assert (_DELTA.size, _QK_NORM.size) == (ctypes.sizeof(_DeltaProblem), ctypes.sizeof(_QkNormProblem))


def _signatures():
    VP, SZ = ctypes.c_void_p, ctypes.c_size_t   # a problem is passed by its address
    return {
        "kata_fwd_delta_workspace_size": (SZ, [VP]),
        "kata_fwd_delta": (_I32, [VP] * 11 + [SZ, VP]),
        "kata_bwd_delta_workspace_size": (SZ, [VP]),
        "kata_bwd_delta": (_I32, [VP] * 17 + [SZ, VP]),
        "kata_decode_delta": (_I32, [VP] * 9),
        "kata_fwd_qk_norm": (_I32, [VP] * 11),
        "kata_bwd_qk_norm_workspace_size": (SZ, [VP]),
        "kata_bwd_qk_norm": (_I32, [VP] * 15 + [SZ, VP]),
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
    operands that come out of them are kept in two terms (2^-18), with return_state in three, so that outputs may
    differ by a rounding from a call without it.
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


# ---- norms of queries and keys -------------------------------------------------------------------

def _qk_norm_problem(q, k, wq, wk, eps, l2, rates, positions, offset, interleaved, magnitude, axes, outs, grads):
    """The packed kata_qk_norm_problem of a call and the address of its positions, the arguments checked.
    outs: the outputs (None: contiguous ones); grads: dq and dk, or None."""
    device, dtype, shape = q.device, q.dtype, q.shape
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    if len(shape) != 4:
        raise ValueError("q and k must be 4-D (B, T, H, D)")
    B, T, H, D = shape
    Hk = 0
    if k is not None:
        if k.dim() != 4 or k.shape != (B, T, k.shape[2], D) or k.dtype != dtype or k.device != device:
            raise ValueError("q and k must be 4-D (B, T, H, D) and share B, T, D, dtype and device")
        Hk = k.shape[2]
    elif wk is not None:
        raise ValueError("a weight of keys needs k")
    if Hk and not H:
        raise ValueError("k without heads of q: pass it as q")
    w_dtype = None
    if wq is not None:
        if wq.shape != (D,) or not wq.is_contiguous() or wq.device != device:
            raise ValueError(f"q_weight must be a contiguous vector of a head's width on {device}")
        w_dtype = wq.dtype
    if wk is not None:
        if wk.shape != (D,) or not wk.is_contiguous() or wk.device != device:
            raise ValueError(f"k_weight must be a contiguous vector of a head's width on {device}")
        if w_dtype is not None and wk.dtype != w_dtype:
            raise ValueError("the weights must share their dtype")
        w_dtype = wk.dtype
    n, at = 0, None
    pos64 = pos_a = pos_b = pos_t = 0
    n_axes = 1
    if rates is not None:
        n = rates.numel()
        if rates.dim() != 1 or rates.dtype != torch.float64 or not rates.is_contiguous() or rates.device != device:
            raise ValueError(f"rates must be a contiguous fp64 vector on {device}")
        if 2 * n > D:
            raise ValueError("rates turn more coordinates than a head has")
        pos64, n_axes, pos_a, pos_b, pos_t, at = _l._positions(positions, axes, B, T, n, device)
    elif positions is not None or axes is not None:
        raise ValueError("positions need rates")
    tight_q, tight_k = (T * H * D, H * D, D, 1), (T * Hk * D, Hk * D, D, 1)
    sq, sk = q.stride(), tight_k if k is None else k.stride()
    so = [tight_q, tight_k, tight_q, tight_k]        # of the outputs, of the gradients of q' and k'
    for i, given in enumerate((outs, grads)):
        if given is not None:
            so[2 * i] = given[0].stride()
            if k is not None:
                so[2 * i + 1] = given[1].stride()
    if not sq[3] == sk[3] == so[0][3] == so[1][3] == so[2][3] == so[3][3] == 1:
        for x in (q, k, *(outs or ()), *(grads or ())):
            if x is not None:
                _rows_ok(x, "q, k, their outputs and gradients")
    return _QK_NORM.pack(B, T, H, Hk, D, 2 * n, _dtype(dtype), _l._k.KATA_F32 if w_dtype is None else _dtype(w_dtype),
                         1 if interleaved else 0, 1 if l2 else 0, pos64, n_axes, magnitude, eps, pos_a, pos_b, pos_t,
                         offset, *sq[:3], *sk[:3], *so[0][:3], *so[1][:3], *so[2][:3], *so[3][:3]), at


def fwd_qk_norm(q, k, q_weight=None, k_weight=None, eps=1e-6, l2=False, rates=None, positions=None, offset=0,
                interleaved=False, magnitude=1.0, axes=None, out=None):
    """Every head of q and k divided by its size, times a weight, and turned by its position, in one pass:
    z = x / sqrt(mean(x^2) + eps) * weight (l2: the sum in place of the mean, rows of unit length), then the
    turn of rotary() where rates are given, without a rounding in between.

    q (B, T, H, D) and k (B, T, Hk, D) (or None), bf16 or fp32, D up to 256; weights (D,) in fp32, or bf16
    for bf16 rows, or None.  rates, positions, offset, interleaved, magnitude, axes, out: as for rotary().
    Returns the q, or the pair."""
    outs = None
    if out is not None:
        outs = (out,) if torch.is_tensor(out) else tuple(out)
        if len(outs) != (1 if k is None else 2):
            raise ValueError("out must hold an output for each input")
        outs = (*outs, None)[:2]
        for x, y in ((q, outs[0]), (k, outs[1])):
            if x is not None and (y.shape != x.shape or y.dtype != x.dtype or y.device != x.device):
                raise ValueError("out must match the inputs' shapes, dtype and device")
    pr, at = _qk_norm_problem(q, k, q_weight, k_weight, eps, l2, rates, positions, offset, interleaved, magnitude,
                              axes, outs, None)
    oq, ok = (_empty(q), None if k is None else _empty(k)) if outs is None else outs
    if q.numel():
        _run("kata_fwd_qk_norm", q.device, pr, q.data_ptr(), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(rates), at,
             _ptr(axes), oq.data_ptr(), _ptr(ok))
    if outs is not None:
        _written(tuple(x for x in outs if x is not None))
    return oq if k is None else (oq, ok)


def bwd_qk_norm(dq, dk, q, k, q_weight=None, k_weight=None, eps=1e-6, l2=False, rates=None, positions=None, offset=0,
                interleaved=False, magnitude=1.0, axes=None, params=True, workspace=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of sum(dq * q') + sum(dk * k'), q' and k' as fwd_qk_norm
    returns them for the same arguments.  The weights' have the weights' dtype, summed over tokens and heads
    in a fixed order; None without a weight or with params=False."""
    for name, x, y in (("dq", dq, q), ("dk", dk, k)):
        if (x is None) != (y is None) or (x is not None and (x.shape != y.shape or x.dtype != y.dtype or x.device != y.device)):
            raise ValueError(f"{name} must match its input's shape, dtype and device")
    pr, at = _qk_norm_problem(q, k, q_weight, k_weight, eps, l2, rates, positions, offset, interleaved, magnitude,
                              axes, None, (dq, dk))
    gq, gk = _empty(q), None if k is None else _empty(k)
    gw = [_empty(w) if w is not None and params else None for w in (q_weight, k_weight)]
    if q.numel():
        sums = gw[0] is not None or gw[1] is not None
        ws = _workspace(_workspace_size("kata_bwd_qk_norm_workspace_size", pr) if sums else 0, workspace, q.device)
        _run("kata_bwd_qk_norm", q.device, pr, dq.data_ptr(), _ptr(dk), q.data_ptr(), _ptr(k), _ptr(q_weight),
             _ptr(k_weight), _ptr(rates), at, _ptr(axes), gq.data_ptr(), _ptr(gk), _ptr(gw[0]), _ptr(gw[1]), _ptr(ws),
             _bytes(ws))
    else:
        for x in gw:
            if x is not None:
                x.zero_()
    return gq, gk, gw[0], gw[1]


def qk_norm_workspace_size(q, k=None):
    """Bytes of workspace bwd_qk_norm needs for the gradients of weights."""
    return _workspace_size("kata_bwd_qk_norm_workspace_size",
                           _qk_norm_problem(q, k, None, None, 0.0, False, None, None, 0, False, 1.0, None, None, (q, k))[0])


# ---- autograd --------------------------------------------------------------------------------------

class _QkNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, eps, l2, rates, positions, offset, interleaved, magnitude, axes):
        ctx.save_for_backward(q, k, q_weight, k_weight, rates, positions, axes)
        ctx.cfg = dict(eps=eps, l2=l2, offset=offset, interleaved=interleaved, magnitude=magnitude)
        return fwd_qk_norm(q, k, q_weight, k_weight, rates=rates, positions=positions, axes=axes, **ctx.cfg)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk=None):
        q, k, q_weight, k_weight, rates, positions, axes = ctx.saved_tensors
        dq, dk, dwq, dwk = bwd_qk_norm(dq.contiguous(), None if dk is None else dk.contiguous(), q, k, q_weight, k_weight,
                                       rates=rates, positions=positions, axes=axes,
                                       params=ctx.needs_input_grad[2] or ctx.needs_input_grad[3], **ctx.cfg)
        return (dq, dk, dwq if ctx.needs_input_grad[2] else None, dwk if ctx.needs_input_grad[3] else None,
                *[None] * 8)


def qk_norm(q, k, q_weight=None, k_weight=None, eps=1e-6, l2=False, rates=None, positions=None, offset=0,
            interleaved=False, magnitude=1.0, axes=None):
    """fwd_qk_norm with bwd_qk_norm as its gradient under torch autograd."""
    return _QkNorm.apply(q, k, q_weight, k_weight, eps, l2, rates, positions, offset, interleaved, magnitude, axes)


class _Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, beta, log_decay, scale, initial_state, cu_seqlens, return_state):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, beta, log_decay, initial_state, cu_seqlens)
        ctx.scale = scale
        return fwd_delta(q, k, v, beta, log_decay, scale=scale, initial_state=initial_state,
                         return_state=return_state, cu_seqlens=cu_seqlens)

    @staticmethod
    @once_differentiable
    def backward(ctx, dO, dfinal=None):
        q, k, v, beta, log_decay, initial_state, cu_seqlens = ctx.saved_tensors
        dO = torch.zeros_like(v, memory_format=torch.contiguous_format) if dO is None else _l._dense(dO)
        dq, dk, dv, db, dl, dinit = bwd_delta(q, k, v, beta, dO, log_decay, scale=ctx.scale,
                                              initial_state=initial_state, cu_seqlens=cu_seqlens,
                                              dfinal_state=None if dfinal is None else _l._dense(dfinal))
        return dq, dk, dv, db, dl, None, dinit, None, None


def parallel_delta_attn(q, k, v, beta, log_decay=None, scale=1.0, initial_state=None, return_state=False,
                        cu_seqlens=None, qk_norm=None, rotary=None, positions=None, interleaved=False, norm=None):
    """The gated delta rule as a differentiable op, q and k (B, T, Hk, dk), v (B, T, H, dv) -> (B, T, H, dv) (see
    fwd_delta), the output in the inputs' dtype.  All of q, k, v, beta, log_decay and the initial state have
    gradients.

    qk_norm: "l2" (q and k divided to unit length) or (q_weight, k_weight[, eps]) (divided by their root mean
    square, times a weight), see fwd_qk_norm.  rotary: (rates, magnitude) of rotary_rates, with positions of
    several axes (rates, magnitude, axes): q and k are turned by `positions` (with cu_seqlens they must be
    given), behind the norm and in its pass.  norm: (weight, bias[, eps]): the outputs go through a layer norm,
    over each head for a weight of dv elements, over all heads of a token for one of H dv."""
    if rotary is not None and cu_seqlens is not None and positions is None:
        raise ValueError("packed sequences need positions for the rotary turn")
    if qk_norm is not None:
        if qk_norm == "l2":
            wq, wk, eps = None, None, 1e-6
        elif isinstance(qk_norm, (tuple, list)) and len(qk_norm) in (2, 3):
            wq, wk, eps = (*qk_norm, 1e-6)[:3]
        else:
            raise ValueError("qk_norm must be 'l2' or (q_weight, k_weight[, eps])")
        rates, magnitude, axes = (None, 1.0, None) if rotary is None else _l.rotary_table(rotary)
        q, k = _QkNorm.apply(q, k, wq, wk, eps, qk_norm == "l2", rates, positions if rotary is not None else None, 0,
                             interleaved, magnitude, axes)
    elif rotary is not None:
        q, k = _l.turn(q, k, rotary, positions, 0, interleaved)
    got = _Delta.apply(q, k, v, beta, log_decay, scale, initial_state, cu_seqlens, return_state)
    o, final = got if return_state else (got, None)
    if norm is not None:
        o = _l.norm_heads(o, norm)
    return (o, final) if return_state else o
