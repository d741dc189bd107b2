"""CPU fp64 oracle of the decayed linear attention, the rotary positions and the layer norm.

TEST INFRASTRUCTURE ONLY, like kata_oracle: plain definitions in numpy float64, sharing no code with
the GPU package.  Pins (tests/test_layer_oracle.py): decay_closed against the token-by-token
recurrence, its gradients against central differences and against torch float64 autograd, rotary
against complex multiplication and its own inverse, layer_norm's gradients against differences.

Per head (T, d) arrays and a log decay ld, g = exp(ld):
  S_t = g S_{t-1} + k_t v_t^T,  o_t = scale q_t S_t
"""

import numpy as np

__all__ = ["decay_weights", "decay_closed", "decay_recurrent", "decay_backward", "decay_sizes", "rotary",
           "layer_norm", "layer_norm_backward"]


def decay_weights(ld, T):
    """g^(t-s) for s <= t, else 0; g = 0 (ld = -inf) gives the identity."""
    e = np.arange(T)[:, None] - np.arange(T)[None, :]
    with np.errstate(invalid="ignore"):
        w = np.where(e == 0, 1.0, np.exp(ld * np.maximum(e, 0).astype(float)))
    return np.where(e >= 0, w, 0.0)


def _power(ld, n):
    n = np.asarray(n, dtype=float)
    with np.errstate(invalid="ignore"):
        return np.where(n == 0, 1.0, np.exp(ld * n))


def decay_closed(q, k, v, ld, scale=1.0, S0=None):
    """(o, final state) of one head."""
    T = q.shape[0]
    A = decay_weights(ld, T) * (q @ k.T)
    o = A @ v
    left = _power(ld, T - 1 - np.arange(T))
    S = (k * left[:, None]).T @ v
    if S0 is not None:
        o = o + _power(ld, np.arange(T) + 1)[:, None] * (q @ S0)
        S = S + _power(ld, T) * S0
    return scale * o, S


def decay_recurrent(q, k, v, ld, scale=1.0, S0=None):
    g = float(np.exp(ld))
    S = np.zeros((q.shape[1], v.shape[1])) if S0 is None else S0.copy()
    out = []
    for t in range(q.shape[0]):
        S = g * S + np.outer(k[t], v[t])
        out.append(scale * (q[t] @ S))
    return np.array(out).reshape(q.shape[0], v.shape[1]), S


def decay_backward(q, k, v, dO, ld, scale=1.0, S0=None, dS=None):
    """(dq, dk, dv, dS0) of sum(dO * o) + sum(dS * final state), by the derivative of the closed form."""
    T = q.shape[0]
    W = decay_weights(ld, T)
    dA = scale * W * (dO @ v.T)
    dq = dA @ k
    dk = dA.T @ q
    dv = (scale * W * (q @ k.T)).T @ dO
    S0 = np.zeros((q.shape[1], v.shape[1])) if S0 is None else S0
    up = _power(ld, np.arange(T) + 1)[:, None]
    dq = dq + scale * up * (dO @ S0.T)
    dS0 = scale * (q * up).T @ dO
    if dS is not None:
        left = _power(ld, T - 1 - np.arange(T))[:, None]
        dk = dk + left * (v @ dS.T)
        dv = dv + left * (k @ dS)
        dS0 = dS0 + _power(ld, T) * dS
    return dq, dk, dv, dS0


def decay_sizes(q, k, v, ld, scale=1.0, S0=None):
    """Sums of absolute terms: (of o, of the final state).  Rounding errors are bounded by multiples
    of them."""
    S0 = None if S0 is None else np.abs(S0)
    T = q.shape[0]
    A = decay_weights(ld, T) * (np.abs(q) @ np.abs(k).T)
    o = A @ np.abs(v)
    S = (np.abs(k) * _power(ld, T - 1 - np.arange(T))[:, None]).T @ np.abs(v)
    if S0 is not None:
        o = o + _power(ld, np.arange(T) + 1)[:, None] * (np.abs(q) @ S0)
        S = S + _power(ld, T) * S0
    return abs(scale) * o, S


def rotary(x, positions, rates, interleaved=False, magnitude=1.0, inverse=False):
    """x (B, T, H, D), positions (B, T)."""
    n = len(rates)
    angle = positions[..., None, None].astype(float) * np.asarray(rates) * (-1.0 if inverse else 1.0)
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y = x.astype(float).copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[..., None]
    y = y if w is None else y * w
    return (y if b is None else y + b), mean, rstd


def layer_norm_backward(dy, x, w=None, eps=1e-5):
    _, mean, rstd = layer_norm(x, eps=eps)
    hat = (x - mean[..., None]) * rstd[..., None]
    t = dy if w is None else dy * w
    dx = rstd[..., None] * (t - t.mean(-1, keepdims=True) - hat * (t * hat).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    return dx, (dy * hat).sum(lead), dy.sum(lead)
