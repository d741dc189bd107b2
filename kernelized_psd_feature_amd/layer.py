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
import functools
import math
import struct

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version as _written   # tensors that a kernel has written

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


# The same layouts for struct.pack: a call of a few microseconds is mostly spent in its arguments.
_DECAY = struct.Struct("8if15q")
_ROTARY = struct.Struct("10if15q")
_NORM = struct.Struct("q3if4q")
assert (_DECAY.size, _ROTARY.size, _NORM.size) == tuple(
    ctypes.sizeof(x) for x in (_DecayProblem, _RotaryProblem, _NormProblem))


def _signatures():
    VP, SZ = ctypes.c_void_p, ctypes.c_size_t   # a problem is passed by its address
    return {
        "kata_fwd_decay_workspace_size": (SZ, [VP]),
        "kata_fwd_decay": (_I32, [VP] * 10 + [SZ, VP]),
        "kata_bwd_decay_workspace_size": (SZ, [VP]),
        "kata_bwd_decay": (_I32, [VP] * 14 + [SZ, VP]),
        "kata_decode_decay": (_I32, [VP] * 8),
        "kata_rotary": (_I32, [VP] * 8),
        "kata_rotary_axes": (_I32, [VP] * 6 + [_I32, _I64] + [VP] * 3),
        "kata_fwd_layer_norm": (_I32, [VP] * 8),
        "kata_bwd_layer_norm_workspace_size": (SZ, [VP]),
        "kata_bwd_layer_norm": (_I32, [VP] * 10 + [SZ, VP]),
    }


# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(name, device, *args):
    """One entry point on the device's current stream."""
    fn, index = getattr(_k._LIB or _k._lib(), name), device.index
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status:
        _k._check(status, name)


@functools.lru_cache(maxsize=1024)
def _workspace_size(name, problem):
    return int(getattr(_k._lib(), name)(problem))


def _ptr(x):
    return None if x is None else x.data_ptr()


def _rows_ok(x, name):
    if x.stride(-1) != 1 and x.shape[-1] > 1 and x.numel():
        raise ValueError(f"{name}: last dimension must be contiguous")
    return x.stride()[:3]


def _same_device(device, *named):
    for name, x in named:
        if x is not None and x.device != device:
            raise ValueError(f"{name} must be on {device}")


def _empty(x):
    """A new contiguous tensor like x."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty_like(x, memory_format=torch.contiguous_format)


_DTYPES = {torch.float32: _k.KATA_F32, torch.bfloat16: _k.KATA_BF16}


def _dtype(dt):
    code = _DTYPES.get(dt)
    return _k._dtype_code(dt) if code is None else code


def _workspace(need, given, device):
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if given.device != device or not given.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    return given


def _bytes(x):
    return 0 if x is None else x.numel() * x.element_size()


# ---- linear attention with one decay per head -------------------------------------------------

def _decay_problem(q, k, v, log_decay, scale, cu_seqlens, o=None, dO=None, zero_tail=0):
    """The packed kata_decay_problem of a call, its arguments checked."""
    device, dtype, shape = q.device, q.dtype, q.shape
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    if len(shape) != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be 4-D (B, T, H, D)")
    B, T, H, dk = shape
    dv = v.shape[3]
    if k.shape != shape or v.shape != (B, T, H, dv) or k.dtype != dtype or v.dtype != dtype:
        raise ValueError("q, k, v must share (B, T, H) and dtype; q and k share dk")
    if log_decay.shape != (H,) or log_decay.dtype != torch.float32 or not log_decay.is_contiguous():
        raise ValueError("log_decay must be a contiguous fp32 tensor of shape (H,)")
    if k.device != device or v.device != device or log_decay.device != device \
            or (o is not None and o.device != device):
        raise ValueError(f"k, v, log_decay and out must be on {device}")
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
    return _DECAY.pack(n, H, T, dk, dv, packed, zero_tail, _dtype(dtype), scale, *sq[:3], *sk[:3], *sv[:3],
                       *so[:3], *sdo[:3])


def decay_state_shape(q, v, cu_seqlens=None):
    """Shape of the states of (B, T, H, dk) queries and (B, T, H, dv) values: (n, H, dk, dv) fp32 for
    n sequences."""
    n = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    return (n, q.shape[2], q.shape[3], v.shape[3])


def _state(x, shape, device, name):
    if x is not None and (x.shape != shape or x.dtype != torch.float32 or not x.is_contiguous()
                          or x.device != device):
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {shape} on {device}")
    return x


def _out_like(v, out):
    if out is None:
        return _empty(v)
    if out.shape != v.shape or out.dtype != v.dtype or out.device != v.device:
        raise ValueError("out must match v's shape, dtype and device")
    return out


def fwd_decay(q, k, v, log_decay, scale=1.0, initial_state=None, return_state=False,
              cu_seqlens=None, out=None, workspace=None):
    """o_t = scale q_t S_t with S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, in chunks (MFMA).

    q, k (B, T, H, dk), v (B, T, H, dv), bf16 or fp32, widths up to 128 with rows of whole 16 bytes,
    any (b, t, h) strides that keep rows apart, or zero (broadcast axes); o has the inputs' dtype.  log_decay: fp32 (H,).
    cu_seqlens: int32 (n + 1,) offsets of n sequences packed into B = 1; rows of no sequence are zero
    in a new output and left as they are in `out`, which must not overlap an input.
    initial_state, and the final state with return_state: fp32 (n, H, dk, dv); a state that is returned
    has its terms added exactly, so bf16 outputs may differ from a call without it by a rounding.
    Sums and states are fp32.  bf16 operands of a product are rounded: the state that a chunk of 64
    tokens starts from, and the weight of a pair of tokens behind the first 512 rows of a sequence where
    exp(2 log_decay) >= 3/4; with the output's own rounding that is a relative error of 1.7e-3 to
    2.3e-3.  fp32 inputs have none of these roundings.
    workspace: uint8, decay_workspace_size() bytes (allocated here otherwise)."""
    o = _out_like(v, out)
    pr = _decay_problem(q, k, v, log_decay, scale, cu_seqlens, o=o, zero_tail=1 if out is None else 0)
    shape, device = decay_state_shape(q, v, cu_seqlens), q.device
    _state(initial_state, shape, device, "initial_state")
    final = torch.empty(shape, dtype=torch.float32, device=device) if return_state else None
    if q.shape[0] * q.shape[1] == 0:
        if final is not None:
            final.copy_(initial_state) if initial_state is not None else final.zero_()
    elif q.shape[2]:
        ws = _workspace(_workspace_size("kata_fwd_decay_workspace_size", pr), workspace, device)
        _run("kata_fwd_decay", device, pr, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
             _ptr(cu_seqlens), _ptr(initial_state), o.data_ptr(), _ptr(final), _ptr(ws), _bytes(ws))
    if out is not None:
        _written(out)
    return (o, final) if return_state else o


def decay_workspace_size(q, k, v, log_decay, cu_seqlens=None, backward=False):
    """Bytes of workspace fwd_decay (or bwd_decay) needs."""
    return _workspace_size(f"kata_{'bwd' if backward else 'fwd'}_decay_workspace_size",
                           _decay_problem(q, k, v, log_decay, 1.0, cu_seqlens))


def bwd_decay(q, k, v, dO, log_decay, scale=1.0, initial_state=None, dfinal_state=None,
              cu_seqlens=None, workspace=None):
    """Gradients (dq, dk, dv, dinitial_state) of sum(dO * o) + sum(dfinal_state * final_state), the
    first three in the inputs' dtype, the last one fp32 (None without an initial_state).  Rows of no
    packed sequence get zeros.  bf16 operands are rounded as in fwd_decay; for dk and dv the first rows
    are a sequence's last ones."""
    if dO.shape != v.shape or dO.dtype != q.dtype:
        raise ValueError("dO must match v's shape and q's dtype")
    pr = _decay_problem(q, k, v, log_decay, scale, cu_seqlens, dO=dO, zero_tail=1)
    shape, device = decay_state_shape(q, v, cu_seqlens), q.device
    _state(initial_state, shape, device, "initial_state")
    _state(dfinal_state, shape, device, "dfinal_state")
    dq, dk, dv = _empty(q), _empty(k), _empty(v)
    dinit = torch.empty(shape, dtype=torch.float32, device=device) if initial_state is not None else None
    if q.shape[0] * q.shape[1] == 0:
        if dinit is not None:
            dinit.copy_(dfinal_state) if dfinal_state is not None else dinit.zero_()
    elif q.shape[2]:
        ws = _workspace(_workspace_size("kata_bwd_decay_workspace_size", pr), workspace, device)
        _run("kata_bwd_decay", device, pr, q.data_ptr(), k.data_ptr(), v.data_ptr(), dO.data_ptr(),
             log_decay.data_ptr(), _ptr(cu_seqlens), _ptr(initial_state), _ptr(dfinal_state),
             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(dinit), _ptr(ws), _bytes(ws))
    return dq, dk, dv, dinit


def decode_decay(q, k, v, log_decay, state, scale=1.0, out=None):
    """Advances `state` (fp32 (B, H, dk, dv), in place) over the T tokens of q, k, v one at a time and
    returns o; T = 1 is one decode step.  All arithmetic is fp32."""
    o = _out_like(v, out)
    pr = _decay_problem(q, k, v, log_decay, scale, None, o=o)
    if state is None:
        raise ValueError("decode_decay needs a state")
    _state(state, decay_state_shape(q, v), q.device, "state")
    if v.numel():
        _run("kata_decode_decay", q.device, pr, q.data_ptr(), k.data_ptr(), v.data_ptr(),
             log_decay.data_ptr(), state.data_ptr(), o.data_ptr())
    _written(state if out is None else (state, out))
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


def rotary_axes(sections, interleaved=False, device="cuda"):
    """Which axis each pair of coordinates turns by, for positions with several axes: an int32 vector of
    sum(sections) pairs, sections[a] of them for axis a, one section behind the other, or with interleaved
    dealt out in turn while a section has some left."""
    if not sections or any(n < 0 for n in sections):
        raise ValueError("sections must be counts of pairs, one for each axis")
    axes = [a for a, n in enumerate(sections) for _ in range(n)]
    if interleaved:
        axes = [a for i in range(max(sections)) for a, n in enumerate(sections) if i < n]
    return torch.tensor(axes, dtype=torch.int32).to(device)


def _positions(positions, axes, B, T, pairs, device):
    """(pos64, axes, stride of the axes, of b, of t, address) of positions that broadcast to (B, T), or with
    axes to (axes, B, T)."""
    if positions is None:
        if axes is not None:
            raise ValueError("several axes need positions")
        return 0, 1, 0, 0, 0, None
    if positions.dtype not in (torch.int32, torch.int64) or positions.device != device:
        raise ValueError(f"positions must be int32 or int64 on {device}")
    pos64 = int(positions.dtype == torch.int64)
    if axes is None:
        try:
            x = positions if positions.shape == (B, T) else positions.expand(B, T)
        except RuntimeError:
            raise ValueError("positions must broadcast to (B, T)") from None
        return pos64, 1, 0, *x.stride(), positions.data_ptr()
    if axes.shape != (pairs,) or axes.dtype != torch.int32 or not axes.is_contiguous() or axes.device != device:
        raise ValueError(f"axes must be a contiguous int32 vector of an axis for each rate on {device}")
    shape = positions.shape
    try:
        x = None if len(shape) != 3 or not shape[0] else positions if shape[1:] == (B, T) else positions.expand(shape[0], B, T)
    except RuntimeError:
        x = None
    if x is None:
        raise ValueError("positions must broadcast to (axes, B, T)")
    return pos64, x.shape[0], *x.stride(), positions.data_ptr()


def rotary(q, k, rates, positions=None, offset=0, interleaved=False, magnitude=1.0, inverse=False,
           out=None, axes=None):
    """q and k turned by their positions in one launch: the first 2 * len(rates) coordinates of every
    head, as pairs (i, i + len(rates)), or neighbours with interleaved; the others are copied.

    q (B, T, H, D) and k (B, T, Hk, D) (or None), bf16 or fp32; positions: int32 or int64, broadcastable
    to (B, T), or None: offset + t.  axes (rotary_axes): positions have several axes, (axes, B, T), and pair i
    turns by that of axis axes[i].  inverse negates the angles: the gradient.  out: outputs of q (and
    k), which may be q and k themselves and overlap neither otherwise.  Returns the turned q, or the pair."""
    device, dtype, shape = q.device, q.dtype, q.shape
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    if len(shape) != 4:
        raise ValueError("q and k must be 4-D (B, T, H, D)")
    B, T, H, D = shape
    n = rates.numel()
    if rates.dim() != 1 or rates.dtype != torch.float64 or not rates.is_contiguous() or rates.device != device:
        raise ValueError(f"rates must be a contiguous fp64 vector on {device}")
    if 2 * n > D:
        raise ValueError("rates turn more coordinates than a head has")
    if out is None:
        oq, ok = _empty(q), None if k is None else _empty(k)
    else:
        outs = (out,) if torch.is_tensor(out) else tuple(out)
        if len(outs) != (1 if k is None else 2):
            raise ValueError("out must hold an output for each input")
        oq, ok = (*outs, None)[:2]
        for x, y in ((q, oq), (k, ok)):
            if x is not None and (y.shape != x.shape or y.dtype != dtype or y.device != device):
                raise ValueError("out must match the inputs' shapes, dtype and device")
    sq, soq, Hk, pk, pok = q.stride(), oq.stride(), 0, None, None
    sk, sok = sq, soq
    if k is not None:
        if k.dim() != 4 or k.shape != (B, T, k.shape[2], D) or k.dtype != dtype or k.device != device:
            raise ValueError("q and k must be 4-D (B, T, H, D) and share B, T, D, dtype and device")
        Hk, sk, sok, pk, pok = k.shape[2], k.stride(), ok.stride(), k.data_ptr(), ok.data_ptr()
    if not sq[3] == sk[3] == soq[3] == sok[3] == 1:
        for name, x in (("q", q), ("k", k), ("out", oq), ("out", ok)):
            if x is not None:
                _rows_ok(x, name)
    pos64, n_axes, pos_a, pos_b, pos_t, at = _positions(positions, axes, B, T, n, device)
    pq, poq = q.data_ptr(), oq.data_ptr()
    if H == 0 and Hk:                                # only k has heads: its turn is a call of one tensor
        H, sq, soq, pq, poq, Hk = Hk, sk, sok, pk, pok, 0
    if B * T * H * D:
        pr = _ROTARY.pack(B, T, H, Hk, D, 2 * n, _dtype(dtype), 1 if interleaved else 0, 1 if inverse else 0,
                          pos64, magnitude, pos_b, pos_t, offset, *sq[:3], *sk[:3], *soq[:3], *sok[:3])
        if axes is None or n == 0:                   # (no pairs: no axis is looked at, and axes has no address)
            _run("kata_rotary", device, pr, pq, pk, rates.data_ptr(), at, poq, pok)
        else:
            _run("kata_rotary_axes", device, pr, pq, pk, rates.data_ptr(), at, axes.data_ptr(), n_axes, pos_a, poq, pok)
    if out is not None:
        _written(outs)
    return oq if k is None else (oq, ok)


# ---- layer norm --------------------------------------------------------------------------------

def _rows(x):
    """x as (rows, N) with one row stride, copied only where its axes do not collapse or its rows overlap
    (windows of one array)."""
    N = x.shape[-1]
    if x.dim() == 2:
        y = x
    else:
        try:
            y = x.view(-1, N)
        except RuntimeError:
            return x.contiguous().view(-1, N)
    step, one = y.stride()
    return y if (one == 1 or N == 1) and (step >= N or step == 0 or y.shape[0] == 1) else y.contiguous()


def _check_norm(x, weight, bias):
    """The weights' dtype code, the arguments checked."""
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    shape, device, dt = x.shape, x.device, None
    if not shape or shape[-1] < 1:
        raise ValueError("x needs a last axis of at least one element")
    if weight is not None:
        dt = weight.dtype
        if weight.shape != shape[-1:] or not weight.is_contiguous() or weight.device != device:
            raise ValueError(f"weight must be a contiguous vector of the last axis's length on {device}")
    if bias is not None:
        if bias.shape != shape[-1:] or not bias.is_contiguous() or bias.device != device:
            raise ValueError(f"bias must be a contiguous vector of the last axis's length on {device}")
        if dt is not None and bias.dtype != dt:
            raise ValueError("weight and bias must share their dtype")
        dt = bias.dtype
    return _k.KATA_F32 if dt is None else _dtype(dt)


def fwd_layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, return_stats=False):
    """Layer norm over the last axis of x (bf16 or fp32, any leading axes); weight and bias (N,) in
    fp32, or bf16 for bf16 rows.  With return_stats also the rows' mean and 1 / sqrt(var + eps), fp32
    of x's leading shape, for bwd_layer_norm.  out may be x."""
    wt = _check_norm(x, weight, bias)
    device, dtype, shape, N, mean, rstd = x.device, x.dtype, x.shape, x.shape[-1], None, None
    if out is None:
        y = _empty(x)
        y2_stride = N
    else:
        y = out
        if out.shape != shape or out.dtype != dtype or out.device != device:
            raise ValueError("out must match x's shape, dtype and device")
        try:
            y2 = y.view(-1, N)
        except RuntimeError:
            raise ValueError("out's leading axes must collapse into one") from None
        if N > 1 and y2.stride(1) != 1:
            raise ValueError("out: last dimension must be contiguous")
        y2_stride = y2.stride(0)
    if return_stats:
        mean, rstd = (torch.empty(shape[:-1], dtype=torch.float32, device=device) for _ in range(2))
    if y.numel():
        x2 = _rows(x)
        pr = _NORM.pack(x2.shape[0], N, _dtype(dtype), wt, eps, x2.stride(0), N, y2_stride, N)
        _run("kata_fwd_layer_norm", device, pr, x2.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(),
             _ptr(mean), _ptr(rstd))
    if out is not None:
        _written(out)
    return (y, mean, rstd) if return_stats else y


def layer_norm_workspace_size(x, weight=None):
    """Bytes of workspace bwd_layer_norm needs for the gradients of the weight and the bias."""
    wt, N = _check_norm(x, weight, None), x.shape[-1]
    return _workspace_size("kata_bwd_layer_norm_workspace_size",
                           _NORM.pack(x.numel() // N, N, _dtype(x.dtype), wt, 0.0, N, N, N, N))


def bwd_layer_norm(dy, x, weight, mean, rstd, params=True, workspace=None):
    """Gradients (dx, dweight, dbias) of sum(dy * y), mean and rstd as fwd_layer_norm returned them.
    dweight and dbias have the weight's dtype (fp32 without one), summed over the rows in a fixed
    order; None with params=False."""
    wt = _check_norm(x, weight, None)
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must match x's shape and dtype")
    for name, s in (("mean", mean), ("rstd", rstd)):
        if s.shape != x.shape[:-1] or s.dtype != torch.float32 or not s.is_contiguous():
            raise ValueError(f"{name} must be a contiguous fp32 tensor of x's leading shape")
    device, N, dw, db = x.device, x.shape[-1], None, None
    _same_device(device, ("dy", dy), ("mean", mean), ("rstd", rstd))
    dx = _empty(x)
    if params:
        dt = weight.dtype if weight is not None else torch.float32
        dw, db = (torch.empty(N, dtype=dt, device=device) for _ in range(2))
    if x.numel():
        x2, g2 = _rows(x), _rows(dy)
        pr = _NORM.pack(x2.shape[0], N, _dtype(x.dtype), wt, 0.0, x2.stride(0), g2.stride(0), N, N)
        ws = _workspace(_workspace_size("kata_bwd_layer_norm_workspace_size", pr) if params else 0,
                        workspace, device)
        _run("kata_bwd_layer_norm", device, pr, g2.data_ptr(), x2.data_ptr(), _ptr(weight), mean.data_ptr(),
             rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(ws), _bytes(ws))
    elif params:
        dw.zero_(), db.zero_()
    return dx, dw, db


# ---- autograd ----------------------------------------------------------------------------------

def _dense(x):
    """A gradient as the kernels read it: contiguous, on a 16-byte boundary (a concatenation's gradient
    comes as a view at any element)."""
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


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
        dO = torch.zeros_like(v, memory_format=torch.contiguous_format) if dO is None else _dense(dO)
        dq, dk, dv, dinit = bwd_decay(q, k, v, dO, log_decay, scale=ctx.scale,
                                      initial_state=initial_state, cu_seqlens=cu_seqlens,
                                      dfinal_state=None if dfinal is None else _dense(dfinal))
        return dq, dk, dv, None, None, dinit, None, None


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, rates, positions, offset, interleaved, magnitude, axes):
        ctx.save_for_backward(rates, positions, axes)
        ctx.cfg = (offset, interleaved, magnitude)
        return rotary(q, k, rates, positions, offset, interleaved, magnitude, axes=axes)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        rates, positions, axes = ctx.saved_tensors
        offset, interleaved, magnitude = ctx.cfg
        dq, dk = rotary(dq.contiguous(), dk.contiguous(), rates, positions, offset, interleaved,
                        magnitude, inverse=True, axes=axes)
        return dq, dk, None, None, None, None, None, None


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


def rotary_table(table):
    """(rates, magnitude, axes) of a layer's rotary argument: (rates, magnitude) as rotary_rates returns them, with
    positions of several axes (rates, magnitude, axes)."""
    if not isinstance(table, (tuple, list)) or len(table) not in (2, 3):
        raise ValueError("rotary must be (rates, magnitude) or (rates, magnitude, axes)")
    return (*table, None)[:3]


def turn(q, k, table, positions=None, offset=0, interleaved=False):
    """rotary() under torch autograd; table: see rotary_table()."""
    rates, magnitude, axes = rotary_table(table)
    return _Rotary.apply(q, k, rates, positions, offset, interleaved, magnitude, axes)


def norm_heads(o, norm):
    """Layer norm of (B, T, H, dv) outputs; norm: (weight, bias[, eps]), over each head for a weight of dv elements,
    over all heads of a token for one of H dv."""
    weight, bias, eps = (*norm, 1e-5)[:3]
    H, dv = o.shape[2:]
    n = weight.numel() if weight is not None else dv
    if n < 1 or n not in (dv, H * dv):
        raise ValueError("the norm's weight must have dv or H * dv elements")
    return layer_norm(o.reshape(*o.shape[:2], H * dv // n, n), weight, bias, eps).reshape(o.shape)


def parallel_decay_attn(q, k, v, log_decay, scale=1.0, initial_state=None, return_state=False,
                        cu_seqlens=None, rotary=None, positions=None, interleaved=False, norm=None):
    """Linear attention with one decay per head as a differentiable op, (B, T, H, dk) -> (B, T, H, dv)
    (see fwd_decay), the output in the inputs' dtype.

    rotary: (rates, magnitude) of rotary_rates, with positions of several axes (rates, magnitude, axes): q and k
    are turned first, by `positions` (see rotary(); with cu_seqlens they must be given).  norm: (weight, bias[, eps]): the outputs go through a layer
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
        o = norm_heads(o, norm)
    return (o, final) if return_state else o
