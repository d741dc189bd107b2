"""Linear attention with one decay per head, rotary positions and layer norm: the binding of the
second part of include/kata.h.  Like the rest of the package it marshals torch tensors into the C
ABI and enqueues the work on the current stream of the tensors' device.

    o = fwd_decay(q, k, v, log_decay)                     # chunked form, batch or packed
    dq, dk, dv, dstate = bwd_decay(q, k, v, dO, log_decay)
    o = decode_decay(q, k, v, log_decay, state)           # recurrent form, state in place
    q, k = rotary(q, k, rates, positions=positions)       # rates, m = rotary_rates(64)
    y = fwd_layer_norm(x, weight, bias)                   # bwd_layer_norm: its gradients
    o = parallel_decay_attn(q, k, v, log_decay, rotary=(rates, m), norm=(weight, bias))

The last one and layer_norm are differentiable by torch autograd.
"""

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

import kernelized_psd_feature_amd as _k

_I32, _I64, _F32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class _DecayProblem(ctypes.Structure):
    _fields_ = [("n_seq", _I32), ("H", _I32), ("T", _I32), ("dk", _I32), ("dv", _I32),
                ("packed", _I32), ("zero_tail", _I32), ("dtype", _I32), ("scale", _F32),
                ("sq", _I64 * 3), ("sk", _I64 * 3), ("sv", _I64 * 3), ("so", _I64 * 3),
                ("sdo", _I64 * 3)]


class _RotaryProblem(ctypes.Structure):
    _fields_ = [("B", _I32), ("T", _I32), ("H", _I32), ("Hk", _I32), ("D", _I32), ("rot", _I32),
                ("dtype", _I32), ("interleaved", _I32), ("inverse", _I32), ("pos64", _I32),
                ("magnitude", _F32), ("pos_b", _I64), ("pos_t", _I64), ("offset", _I64),
                ("sq", _I64 * 3), ("sk", _I64 * 3), ("soq", _I64 * 3), ("sok", _I64 * 3)]


class _NormProblem(ctypes.Structure):
    _fields_ = [("rows", _I64), ("N", _I32), ("dtype", _I32), ("w_dtype", _I32), ("eps", _F32),
                ("sx", _I64), ("sdy", _I64), ("sy", _I64), ("sdx", _I64)]


def _signatures():
    VP, SZ = ctypes.c_void_p, ctypes.c_size_t
    D, R, N = (ctypes.POINTER(x) for x in (_DecayProblem, _RotaryProblem, _NormProblem))
    return {
        "kata_fwd_decay_workspace_size": (SZ, [D]),
        "kata_fwd_decay": (_I32, [D] + [VP] * 9 + [SZ, VP]),
        "kata_bwd_decay_workspace_size": (SZ, [D]),
        "kata_bwd_decay": (_I32, [D] + [VP] * 13 + [SZ, VP]),
        "kata_decode_decay": (_I32, [D] + [VP] * 7),
        "kata_rotary": (_I32, [R] + [VP] * 7),
        "kata_fwd_layer_norm": (_I32, [N] + [VP] * 7),
        "kata_bwd_layer_norm_workspace_size": (SZ, [N]),
        "kata_bwd_layer_norm": (_I32, [N] + [VP] * 9 + [SZ, VP]),
    }


def _strides(x, name):
    """Element strides of the (b, t, h) axes; an axis of one entry counts as zero."""
    if x.dim() != 4:
        raise ValueError(f"{name} must be 4-D (B, T, H, D)")
    if x.shape[3] > 1 and x.stride(3) != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    return tuple(x.stride(i) if x.shape[i] > 1 else 0 for i in range(3))


def _on(device, **tensors):
    for name, x in tensors.items():
        if x is not None and x.device != device:
            raise ValueError(f"{name} must be on {device}")


def _workspace(need, given, device):
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if given.device != device:
        raise ValueError(f"workspace must be on {device}")
    return given


def _bytes(x):
    return 0 if x is None else x.numel() * x.element_size()


# ---- linear attention with one decay per head -------------------------------------------------

def _decay_problem(q, k, v, log_decay, scale, cu_seqlens, o=None, dO=None):
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    for name, x in (("q", q), ("k", k), ("v", v)):
        if x.dim() != 4:
            raise ValueError(f"{name} must be 4-D (B, T, H, D)")
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share (B, T, H) and dtype; q and k share dk")
    B, T, H, dk = q.shape
    if log_decay.shape != (H,) or log_decay.dtype != torch.float32 or not log_decay.is_contiguous():
        raise ValueError("log_decay must be a contiguous fp32 tensor of shape (H,)")
    _on(q.device, k=k, v=v, log_decay=log_decay, cu_seqlens=cu_seqlens, out=o, dO=dO)
    pr = _DecayProblem()
    pr.n_seq, pr.H, pr.T, pr.dk, pr.dv = B, H, T, dk, v.shape[3]
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or cu_seqlens.dtype != torch.int32 \
                or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous int32 tensor of n + 1 >= 2 offsets")
        if B != 1:
            raise ValueError("packed sequences lie in one batch row: B must be 1")
        pr.packed, pr.n_seq = 1, cu_seqlens.numel() - 1
    pr.dtype, pr.scale = _k._dtype_code(q.dtype), scale
    pr.sq[:], pr.sk[:], pr.sv[:] = _strides(q, "q"), _strides(k, "k"), _strides(v, "v")
    pr.so[:] = _strides(o, "out") if o is not None else (T * H * pr.dv, H * pr.dv, pr.dv)
    if dO is not None:
        pr.sdo[:] = _strides(dO, "dO")
    return pr


def decay_state_shape(q, v, cu_seqlens=None):
    """Shape of the states of (B, T, H, dk) queries and (B, T, H, dv) values: (n, H, dk, dv) fp32 for
    n sequences."""
    n = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    return (n, q.shape[2], q.shape[3], v.shape[3])


def _state(x, shape, device, name):
    if x is not None and (tuple(x.shape) != shape or x.dtype != torch.float32 or not x.is_contiguous()
                          or x.device != device):
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {shape} on {device}")
    return x


def _out_like(v, out, name="out"):
    if out is None:
        return torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if out.shape != v.shape or out.dtype != v.dtype or out.device != v.device:
        raise ValueError(f"{name} must match v's shape, dtype and device")
    return out


def fwd_decay(q, k, v, log_decay, scale=1.0, initial_state=None, return_state=False,
              cu_seqlens=None, out=None, workspace=None):
    """o_t = scale q_t S_t with S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, in chunks (MFMA).

    q, k (B, T, H, dk), v (B, T, H, dv), bf16 or fp32, widths up to 128 with rows of whole 16 bytes,
    any (b, t, h) strides (broadcast axes too); o has the inputs' dtype.  log_decay: fp32 (H,).
    cu_seqlens: int32 (n + 1,) offsets of n sequences packed into B = 1; rows behind the last one
    are zero in a new output and left as they are in `out`.
    initial_state, and the final state with return_state: fp32 (n, H, dk, dv).
    workspace: uint8, decay_workspace_size() bytes (allocated here otherwise)."""
    o = _out_like(v, out)
    pr = _decay_problem(q, k, v, log_decay, scale, cu_seqlens, o=o)
    shape = decay_state_shape(q, v, cu_seqlens)
    _state(initial_state, shape, q.device, "initial_state")
    final = torch.empty(shape, dtype=torch.float32, device=q.device) if return_state else None
    if q.shape[0] * q.shape[1] == 0:
        if final is not None:
            final.copy_(initial_state) if initial_state is not None else final.zero_()
    elif q.shape[2]:
        pr.zero_tail = 1 if out is None else 0
        lib = _k._lib()
        ws = _workspace(int(lib.kata_fwd_decay_workspace_size(ctypes.byref(pr))), workspace, q.device)
        p = _k._ptr
        with torch.cuda.device(q.device):
            _k._check(lib.kata_fwd_decay(ctypes.byref(pr), p(q), p(k), p(v), p(log_decay),
                                         p(cu_seqlens), p(initial_state), p(o), p(final), p(ws),
                                         _bytes(ws), _k._stream(q.device)), "kata_fwd_decay")
    return (o, final) if return_state else o


def decay_workspace_size(q, k, v, log_decay, cu_seqlens=None, backward=False):
    """Bytes of workspace fwd_decay (or bwd_decay) needs."""
    pr = _decay_problem(q, k, v, log_decay, 1.0, cu_seqlens)
    lib = _k._lib()
    fn = lib.kata_bwd_decay_workspace_size if backward else lib.kata_fwd_decay_workspace_size
    return int(fn(ctypes.byref(pr)))


def bwd_decay(q, k, v, dO, log_decay, scale=1.0, initial_state=None, dfinal_state=None,
              cu_seqlens=None, workspace=None):
    """Gradients (dq, dk, dv, dinitial_state) of sum(dO * o) + sum(dfinal_state * final_state), the
    first three in the inputs' dtype, the last one fp32 (None without an initial_state).  Rows behind
    the last packed sequence get zeros."""
    if dO.shape != v.shape or dO.dtype != q.dtype:
        raise ValueError("dO must match v's shape and q's dtype")
    pr = _decay_problem(q, k, v, log_decay, scale, cu_seqlens, dO=dO)
    pr.zero_tail = 1
    shape = decay_state_shape(q, v, cu_seqlens)
    _state(initial_state, shape, q.device, "initial_state")
    _state(dfinal_state, shape, q.device, "dfinal_state")
    dq, dk, dv = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k, v))
    dinit = torch.empty(shape, dtype=torch.float32, device=q.device) if initial_state is not None else None
    if q.shape[0] * q.shape[1] == 0:
        if dinit is not None:
            dinit.copy_(dfinal_state) if dfinal_state is not None else dinit.zero_()
    elif q.shape[2]:
        lib = _k._lib()
        ws = _workspace(int(lib.kata_bwd_decay_workspace_size(ctypes.byref(pr))), workspace, q.device)
        p = _k._ptr
        with torch.cuda.device(q.device):
            _k._check(lib.kata_bwd_decay(ctypes.byref(pr), p(q), p(k), p(v), p(dO), p(log_decay),
                                         p(cu_seqlens), p(initial_state), p(dfinal_state), p(dq), p(dk),
                                         p(dv), p(dinit), p(ws), _bytes(ws), _k._stream(q.device)),
                      "kata_bwd_decay")
    return dq, dk, dv, dinit


def decode_decay(q, k, v, log_decay, state, scale=1.0, out=None):
    """Advances `state` (fp32 (B, H, dk, dv), in place) over the T tokens of q, k, v one at a time and
    returns o; T = 1 is one decode step.  All arithmetic is fp32."""
    o = _out_like(v, out)
    pr = _decay_problem(q, k, v, log_decay, scale, None, o=o)
    if state is None:
        raise ValueError("decode_decay needs a state")
    _state(state, decay_state_shape(q, v), q.device, "state")
    if q.shape[0] * q.shape[1] * q.shape[2]:
        p = _k._ptr
        with torch.cuda.device(q.device):
            _k._check(_k._lib().kata_decode_decay(ctypes.byref(pr), p(q), p(k), p(v), p(log_decay),
                                                  p(state), p(o), _k._stream(q.device)),
                      "kata_decode_decay")
    return o


# ---- rotary positions --------------------------------------------------------------------------

def rotary_rates(dim, base=10000.0, scaling=None, factor=1.0, original_length=None, low=1.0,
                 high=32.0, device="cuda"):
    """(rates, magnitude) for rotary(): radians a token of the dim / 2 pairs, base^(-2 i / dim), as an
    fp64 tensor, and the factor of the turned coordinates.

    scaling, for contexts `factor` times the trained length:
      None      as trained
      "linear"  every rate divided by factor (positions interpolated)
      "ntk"     base multiplied by factor^(dim / (dim - 2)): the fastest pair keeps its rate, the
                slowest one is divided by factor
      "parts"   by the turns a pair makes over original_length: more than `high` keep their rate,
                fewer than `low` are divided by factor, a ramp in between; magnitude
                0.1 ln(factor) + 1"""
    if dim < 2 or dim % 2:
        raise ValueError("dim must be even and positive")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be positive and factor >= 1")
    if scaling == "ntk":
        if dim == 2:
            raise ValueError("ntk scaling needs dim > 2")
        base = base * factor ** (dim / (dim - 2))
    rates = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    magnitude = 1.0
    if scaling == "linear":
        rates = rates / factor
    elif scaling == "parts":
        if original_length is None or not low < high:
            raise ValueError("parts scaling needs original_length and low < high")
        keep = ((original_length * rates / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        rates = rates / factor * (1 - keep) + rates * keep
        magnitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'parts'")
    return rates.to(device), magnitude


def rotary(q, k, rates, positions=None, offset=0, interleaved=False, magnitude=1.0, inverse=False,
           out=None):
    """q and k turned by their positions in one launch: the first 2 * len(rates) coordinates of every
    head, as pairs (i, i + len(rates)), or neighbours with interleaved; the others are copied.

    q (B, T, H, D) and k (B, T, Hk, D) (or None), bf16 or fp32; positions: int32 or int64, broadcastable
    to (B, T), or None: offset + t.  inverse negates the angles: the gradient.  out: outputs of q (and
    k), which may be q and k themselves.  Returns the turned q, or the pair."""
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    if q.dim() != 4 or (k is not None and (k.dim() != 4 or k.shape[:2] != q.shape[:2] or
                                           k.shape[3] != q.shape[3] or k.dtype != q.dtype)):
        raise ValueError("q and k must be 4-D (B, T, H, D) and share B, T, D and dtype")
    if rates.dim() != 1 or rates.dtype != torch.float64 or not rates.is_contiguous():
        raise ValueError("rates must be a contiguous fp64 vector")
    B, T, H, D = q.shape
    if 2 * rates.numel() > D:
        raise ValueError("rates turn more coordinates than a head has")
    ins = [q] if k is None else [q, k]
    outs = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in ins] if out is None else \
        [out] if torch.is_tensor(out) else list(out)
    if len(outs) != len(ins):
        raise ValueError("out must hold an output for each input")
    for x, y in zip(ins, outs):
        if y.shape != x.shape or y.dtype != x.dtype:
            raise ValueError("out must match the inputs' shapes and dtype")
        _on(q.device, k=x, out=y)
    _on(q.device, rates=rates, positions=positions)
    pr = _RotaryProblem()
    pr.B, pr.T, pr.H, pr.Hk, pr.D, pr.rot = B, T, H, 0 if k is None else k.shape[2], D, 2 * rates.numel()
    pr.dtype, pr.interleaved, pr.inverse = _k._dtype_code(q.dtype), int(interleaved), int(inverse)
    pr.magnitude, pr.offset = magnitude, offset
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("positions must be int32 or int64")
        try:
            at = positions.expand(B, T)
        except RuntimeError:
            raise ValueError("positions must broadcast to (B, T)") from None
        pr.pos64, pr.pos_b, pr.pos_t = int(positions.dtype == torch.int64), at.stride(0), at.stride(1)
    pr.sq[:], pr.soq[:] = _strides(q, "q"), _strides(outs[0], "out")
    if k is not None:
        pr.sk[:], pr.sok[:] = _strides(k, "k"), _strides(outs[1], "out")
    if B * T * H * D and not (k is not None and k.shape[2] == 0):
        p = _k._ptr
        with torch.cuda.device(q.device):
            _k._check(_k._lib().kata_rotary(ctypes.byref(pr), p(q), p(k), p(rates), p(positions),
                                            p(outs[0]), p(outs[1]) if k is not None else None,
                                            _k._stream(q.device)), "kata_rotary")
    return outs[0] if k is None else tuple(outs)


# ---- layer norm --------------------------------------------------------------------------------

def _rows(x):
    """x as (rows, N) with one row stride, copied only where its axes do not collapse."""
    try:
        y = x.view(-1, x.shape[-1])
    except RuntimeError:
        y = x.contiguous().view(-1, x.shape[-1])
    return y if y.shape[1] == 1 or y.stride(1) == 1 else y.contiguous()


def _norm_problem(x, weight, bias, eps):
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs a last axis of at least one element")
    N = x.shape[-1]
    dt = None
    for name, p in (("weight", weight), ("bias", bias)):
        if p is None:
            continue
        if p.shape != (N,) or not p.is_contiguous():
            raise ValueError(f"{name} must be a contiguous vector of the last axis's length")
        if dt is not None and p.dtype != dt:
            raise ValueError("weight and bias must share their dtype")
        dt = p.dtype
    _on(x.device, weight=weight, bias=bias)
    pr = _NormProblem()
    pr.N, pr.eps = N, eps
    pr.dtype = _k._dtype_code(x.dtype)
    pr.w_dtype = _k._dtype_code(dt) if dt is not None else _k.KATA_F32
    return pr


def _row_stride(x2):
    return x2.stride(0) if x2.shape[0] > 1 else x2.shape[1]


def fwd_layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, return_stats=False):
    """Layer norm over the last axis of x (bf16 or fp32, any leading axes); weight and bias (N,) in
    fp32, or bf16 for bf16 rows.  With return_stats also the rows' mean and 1 / sqrt(var + eps), fp32
    of x's leading shape, for bwd_layer_norm.  out may be x."""
    pr = _norm_problem(x, weight, bias, eps)
    if out is not None and (out.shape != x.shape or out.dtype != x.dtype or out.device != x.device):
        raise ValueError("out must match x's shape, dtype and device")
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
    mean, rstd = (torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if return_stats else None
                  for _ in range(2))
    if x.numel():
        x2 = _rows(x)
        try:
            y2 = y.view(-1, pr.N)
        except RuntimeError:
            raise ValueError("out's leading axes must collapse into one") from None
        if pr.N > 1 and y2.stride(1) != 1:
            raise ValueError("out: last dimension must be contiguous")
        pr.rows, pr.sx, pr.sy = x2.shape[0], _row_stride(x2), _row_stride(y2)
        pr.sdy = pr.sdx = pr.N
        p = _k._ptr
        with torch.cuda.device(x.device):
            _k._check(_k._lib().kata_fwd_layer_norm(ctypes.byref(pr), p(x2), p(weight), p(bias), p(y2),
                                                    p(mean), p(rstd), _k._stream(x.device)),
                      "kata_fwd_layer_norm")
    return (y, mean, rstd) if return_stats else y


def layer_norm_workspace_size(x, weight=None):
    """Bytes of workspace bwd_layer_norm needs for the gradients of the weight and the bias."""
    pr = _norm_problem(x, weight, None, 0.0)
    pr.rows = x.numel() // pr.N
    pr.sx = pr.sy = pr.sdy = pr.sdx = pr.N
    return int(_k._lib().kata_bwd_layer_norm_workspace_size(ctypes.byref(pr)))


def bwd_layer_norm(dy, x, weight, mean, rstd, params=True, workspace=None):
    """Gradients (dx, dweight, dbias) of sum(dy * y), mean and rstd as fwd_layer_norm returned them.
    dweight and dbias have the weight's dtype (fp32 without one), summed over the rows in a fixed
    order; None with params=False."""
    pr = _norm_problem(x, weight, None, 0.0)
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must match x's shape and dtype")
    for name, s in (("mean", mean), ("rstd", rstd)):
        if s.shape != x.shape[:-1] or s.dtype != torch.float32 or not s.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 tensor of x's leading shape")
    _on(x.device, dy=dy, mean=mean, rstd=rstd)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dt = weight.dtype if weight is not None else torch.float32
    dw, db = (torch.empty(pr.N, dtype=dt, device=x.device) if params else None for _ in range(2))
    if x.numel():
        x2, g2 = _rows(x), _rows(dy)
        pr.rows, pr.sx, pr.sdy = x2.shape[0], _row_stride(x2), _row_stride(g2)
        pr.sy = pr.sdx = pr.N
        lib, p = _k._lib(), _k._ptr
        ws = _workspace(int(lib.kata_bwd_layer_norm_workspace_size(ctypes.byref(pr))) if params else 0,
                        workspace, x.device)
        with torch.cuda.device(x.device):
            _k._check(lib.kata_bwd_layer_norm(ctypes.byref(pr), p(g2), p(x2), p(weight), p(mean), p(rstd),
                                              p(dx), p(dw), p(db), p(ws), _bytes(ws),
                                              _k._stream(x.device)), "kata_bwd_layer_norm")
    elif params:
        dw.zero_(), db.zero_()
    return dx, dw, db


# ---- autograd ----------------------------------------------------------------------------------

class _Decay(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale, initial_state, cu_seqlens, return_state):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, log_decay, initial_state, cu_seqlens)
        ctx.scale = scale
        return fwd_decay(q, k, v, log_decay, scale=scale, initial_state=initial_state,
                         return_state=return_state, cu_seqlens=cu_seqlens)

    @staticmethod
    @once_differentiable
    def backward(ctx, dO, dfinal=None):
        q, k, v, log_decay, initial_state, cu_seqlens = ctx.saved_tensors
        dO = torch.zeros_like(v, memory_format=torch.contiguous_format) if dO is None else dO.contiguous()
        dq, dk, dv, dinit = bwd_decay(q, k, v, dO, log_decay, scale=ctx.scale,
                                      initial_state=initial_state, cu_seqlens=cu_seqlens,
                                      dfinal_state=None if dfinal is None else dfinal.contiguous())
        return dq, dk, dv, None, None, dinit, None, None


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, rates, positions, offset, interleaved, magnitude):
        ctx.save_for_backward(rates, positions)
        ctx.cfg = (offset, interleaved, magnitude)
        return rotary(q, k, rates, positions, offset, interleaved, magnitude)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        rates, positions = ctx.saved_tensors
        offset, interleaved, magnitude = ctx.cfg
        dq, dk = rotary(dq.contiguous(), dk.contiguous(), rates, positions, offset, interleaved,
                        magnitude, inverse=True)
        return dq, dk, None, None, None, None, None


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = fwd_layer_norm(x, weight, bias, eps, return_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = bias.dtype if bias is not None else None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need_w, need_b = ctx.needs_input_grad[1:3]
        dx, dw, db = bwd_layer_norm(dy, x, weight, mean, rstd, params=need_w or need_b)
        return (dx, dw if need_w else None, db.to(ctx.bias_dtype) if need_b else None, None)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """fwd_layer_norm with bwd_layer_norm as its gradient under torch autograd."""
    return _LayerNorm.apply(x, weight, bias, eps)


def turn(q, k, rotary_table, positions=None, offset=0, interleaved=False):
    """rotary() under torch autograd; rotary_table: (rates, magnitude) as rotary_rates returns them."""
    rates, magnitude = rotary_table
    return _Rotary.apply(q, k, rates, positions, offset, interleaved, magnitude)


def parallel_decay_attn(q, k, v, log_decay, scale=1.0, initial_state=None, return_state=False,
                        cu_seqlens=None, rotary=None, positions=None, interleaved=False, norm=None):
    """Linear attention with one decay per head as a differentiable op, (B, T, H, dk) -> (B, T, H, dv)
    (see fwd_decay), the output in the inputs' dtype.

    rotary: (rates, magnitude) of rotary_rates: q and k are turned first, by `positions` (see rotary();
    with cu_seqlens they must be given).  norm: (weight, bias[, eps]): the outputs go through a layer
    norm, over each head for a weight of dv elements, over all heads of a token for one of H dv.
    log_decay is a constant: it has no gradient, and a tensor that asks for one is refused."""
    if log_decay.requires_grad:
        raise ValueError("log_decay has no gradient: pass it detached")
    if rotary is not None:
        if cu_seqlens is not None and positions is None:
            raise ValueError("packed sequences need positions for the rotary turn")
        q, k = turn(q, k, rotary, positions, 0, interleaved)
    got = _Decay.apply(q, k, v, log_decay, scale, initial_state, cu_seqlens, return_state)
    o, final = got if return_state else (got, None)
    if norm is not None:
        weight, bias, eps = (*norm, 1e-5)[:3]
        n = weight.numel() if weight is not None else v.shape[3]
        if n not in (v.shape[3], v.shape[2] * v.shape[3]):
            raise ValueError("the norm's weight must have dv or H * dv elements")
        o = layer_norm(o.reshape(*o.shape[:2], -1, n), weight, bias, eps).reshape(v.shape)
    return (o, final) if return_state else o
