"""CPU fp64 oracle of the gated delta rule, the norm of queries and keys, and positions of several axes.

TEST INFRASTRUCTURE ONLY, like kata_oracle: plain definitions in numpy float64, sharing no code with the GPU
package.  Pins (tests/test_delta_oracle.py): delta_recurrent against the chunked closed form, its gradients
against central differences and torch float64 autograd, qk_norm against its parts.

Per head (T, d) arrays, b = beta (T,), ld = log decays (T,), g = exp(ld):
  S_t = g_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,  o_t = scale S_t^T q_t
"""

import numpy as np

__all__ = ["delta_recurrent", "delta_backward", "delta_chunked", "delta_sizes", "delta_gradient_sizes", "delta_token_sizes",
           "delta_chunked_backward", "turn", "qk_norm", "qk_norm_backward"]


def _decay(ld):
    with np.errstate(invalid="ignore"):
        return np.exp(np.asarray(ld, dtype=float))


def delta_recurrent(q, k, v, b, ld, scale=1.0, S0=None, keep=False):
    """(o, final state) of one head; with keep also the states behind every token."""
    T = q.shape[0]
    S = np.zeros((q.shape[1], v.shape[1])) if S0 is None else S0.astype(float).copy()
    g, o, states = _decay(ld), np.empty((T, v.shape[1])), []
    for t in range(T):
        S = g[t] * S
        S = S + np.outer(k[t], b[t] * (v[t] - k[t] @ S))
        o[t] = scale * (q[t] @ S)
        if keep:
            states.append(S)
    return (o, S, states) if keep else (o, S)


def delta_backward(q, k, v, b, ld, dO, scale=1.0, S0=None, dS=None):
    """(dq, dk, dv, db, dld, dS0) of sum(dO * o) + sum(dS * final state), token by token backwards."""
    T = q.shape[0]
    _, _, states = delta_recurrent(q, k, v, b, ld, scale, S0, keep=True)
    g = _decay(ld)
    zero = np.zeros((q.shape[1], v.shape[1]))
    first = zero if S0 is None else S0.astype(float)
    D = zero if dS is None else dS.astype(float).copy()
    dq, dk, dv, db, dl = np.empty(q.shape), np.empty(k.shape), np.empty(v.shape), np.empty(T), np.empty(T)
    for t in range(T - 1, -1, -1):
        D = D + scale * np.outer(q[t], dO[t])
        dq[t] = scale * states[t] @ dO[t]
        before = g[t] * (states[t - 1] if t else first)
        err = v[t] - k[t] @ before
        du = k[t] @ D
        db[t] = du @ err
        dv[t] = b[t] * du
        dk[t] = D @ (b[t] * err) - before @ dv[t]
        D = D - np.outer(k[t], dv[t])
        dl[t] = (D * before).sum()
        D = g[t] * D
    return dq, dk, dv, db, dl, D


def delta_chunked(q, k, v, b, ld, scale=1.0, S0=None, C=64):
    """The chunked closed form, by solving (I + A) U = b (V - y K S)."""
    T = q.shape[0]
    S = np.zeros((q.shape[1], v.shape[1])) if S0 is None else S0.astype(float).copy()
    o = np.empty((T, v.shape[1]))
    for t in range(0, T, C):
        Q, K, V, B = q[t:t + C], k[t:t + C], v[t:t + C], b[t:t + C, None]
        c = np.cumsum(ld[t:t + C])
        r = np.exp(np.minimum(c[:, None] - c, 0.0)) * np.tri(len(c))
        y = np.exp(c)[:, None]
        A = B * np.tril(r, -1) * (K @ K.T)
        U = np.linalg.solve(np.eye(len(c)) + A, B * (V - y * (K @ S)))
        o[t:t + C] = scale * (y * (Q @ S) + (r * (Q @ K.T)) @ U)
        S = y[-1] * S + (K * np.exp(c[-1] - c)[:, None]).T @ U
    return o, S


def delta_sizes(q, k, v, b, ld, S0=None):
    """The largest 2-norms along the sequence, per value column, of the state's column and of a token's
    correction and value together (1, dv): what a relative error of an operand is an error of."""
    _, _, states = delta_recurrent(q, k, v, b, ld, 1.0, S0, keep=True)
    states = states + ([] if S0 is None else [S0])
    size = np.max([np.sqrt((s * s).sum(0)) for s in states], 0) if states else np.zeros(v.shape[1])
    return size[None] + (np.abs(v).max(0)[None] if len(v) else 0.0)


def delta_gradient_sizes(q, k, v, b, ld, dO, scale=1.0, S0=None, dS=None, C=64):
    """Sums of absolute terms, per element, of the chunked forms of dq and dk, and per token of the terms that
    dld is a sum of."""
    T = q.shape[0]
    _, _, states = delta_recurrent(q, k, v, b, ld, scale, S0, keep=True)
    zero = np.zeros((q.shape[1], v.shape[1]))
    first = zero if S0 is None else S0
    dv = delta_backward(q, k, v, b, ld, dO, scale, S0, dS)[2]
    o = delta_recurrent(q, k, v, b, ld, scale, S0)[0]
    Bq, Bk, Bl = np.zeros(q.shape), np.zeros(k.shape), np.zeros(T)
    for t in range(0, T, C):
        e = min(T, t + C)
        Q, K, G, dV = np.abs(q[t:e]), np.abs(k[t:e]), np.abs(dO[t:e]), np.abs(dv[t:e])
        S = states[t - 1] if t else first
        D = delta_backward(q[e:], k[e:], v[e:], b[e:], ld[e:], dO[e:], scale, states[e - 1], dS)[5] if e < T else (
            zero if dS is None else dS)
        before = [states[i - 1] if i else first for i in range(t, e)]
        U = np.abs(np.array([b[i] * (v[i] - np.exp(ld[i]) * (k[i] @ s)) for i, s in zip(range(t, e), before)]))
        c = np.cumsum(ld[t:e])
        r = np.exp(np.minimum(c[:, None] - c, 0.0)) * np.tri(len(c))
        y, left = np.exp(c)[:, None], np.exp(c[-1] - c)[:, None]
        PO, PV = abs(scale) * r * (G @ U.T), np.tril(r, -1) * (dV @ U.T)
        Bq[t:e] = abs(scale) * y * (G @ np.abs(S).T) + PO @ K
        Bk[t:e] = left * (U @ np.abs(D).T) + y * (dV @ np.abs(S).T) + PO.T @ Q + PV.T @ K + PV @ K
        terms = (G * np.abs(o[t:e])).sum(1) + (dV * np.abs(v[t:e])).sum(1)
        Bl[t:e] = np.cumsum(terms[::-1])[::-1] + (np.abs(D) * np.abs(states[e - 1])).sum()
    return Bq, Bk, Bl


def delta_token_sizes(q, k, v, b, ld, dO, scale=1.0, S0=None, dS=None):
    """What the roundings of a token's factors are relative to, by token (T,): products of the norms of what is
    multiplied there, for o, dq, dk, dv, db, dld, and for the whole sequence of the final state and dS0.  The state
    and its gradient enter as they are at the token, so the sizes fade with the decays."""
    T, norm = len(q), lambda x: np.sqrt((x * x).sum(-1))  # noqa: E731
    _, S, states = delta_recurrent(q, k, v, b, ld, scale, S0, keep=True)
    g = _decay(ld)
    first = np.zeros((q.shape[1], v.shape[1])) if S0 is None else S0.astype(float)
    D = np.zeros_like(first) if dS is None else dS.astype(float).copy()
    at, before = np.empty(T), np.empty(T)
    for t in range(T - 1, -1, -1):
        D = D + scale * np.outer(q[t], dO[t])
        at[t] = np.linalg.norm(D)
        before[t] = np.linalg.norm(g[t] * (states[t - 1] if t else first))
        D = g[t] * (D - b[t] * np.outer(k[t], k[t] @ D))
    b, nk, nq, s = np.abs(b), norm(k), norm(q), abs(scale)
    err = norm(v) + nk * before
    behind = before * (1 + b * nk * nk) + b * nk * err
    last = np.linalg.norm(S) + (max(behind[-1], np.linalg.norm(first) * g[0] if T == 1 else 0.0) if T else 0.0)
    return dict(o=s * nq * behind, dq=s * norm(dO) * behind, dk=at * b * err + before * b * nk * at, dv=b * nk * at, db=nk * at * err,
                dld=at * before * (1 + b * nk * nk), state=last,
                dS0=np.linalg.norm(D) + (g[0] * at[0] * (1 + b[0] * nk[0] ** 2) if T else 0.0))


def delta_chunked_backward(q, k, v, b, ld, dO, scale=1.0, S0=None, dS=None, C=64, without=""):
    """(dq, dk, dv, db, dld, dS0) by the chunked formulas, without one of their terms where `without` names it:
    dq "state" "pairs"; dk "correction", "state", "scores", "keys", "rows"; dld "state", "read", "write", "pairs"; db
    and dv "inverse" (as if the chunk's tokens had no pairs)."""
    T, names = len(q), [(t, min(t + C, len(q))) for t in range(0, len(q), C)]
    first = np.zeros((q.shape[1], v.shape[1])) if S0 is None else S0.astype(float)
    D = np.zeros_like(first) if dS is None else dS.astype(float).copy()
    entries, S = [], first
    for t, e in names:
        entries.append(S)
        S = delta_recurrent(q[t:e], k[t:e], v[t:e], b[t:e], ld[t:e], scale, S)[1]
    out = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape), np.zeros(T), np.zeros(T)]
    keep = lambda name: 0.0 if name == without else 1.0  # noqa: E731
    for (t, e), S in zip(names[::-1], entries[::-1]):
        Q, K, V, B, G = q[t:e], k[t:e], v[t:e], b[t:e, None], dO[t:e]
        n, c = e - t, np.cumsum(ld[t:e])
        r = np.exp(np.minimum(c[:, None] - c, 0.0)) * np.tri(n)
        y, left = np.exp(c)[:, None], np.exp(c[-1] - c)[:, None]
        A = np.tril(r, -1) * (K @ K.T)
        E = np.linalg.solve(np.eye(n) + A * B.T, V - y * (K @ S))          # U = B E
        U = B * E
        P = scale * r * (Q @ K.T)
        Z = P.T @ G + left * (K @ D)
        X = Z if without == "db inverse" else np.linalg.solve((np.eye(n) + B * A).T, Z)
        dV = B * X
        PO, PV = scale * r * (G @ U.T), -np.tril(r, -1) * (dV @ U.T)
        out[0][t:e] = keep("dq state") * scale * y * (G @ S.T) + keep("dq pairs") * PO @ K
        out[1][t:e] = (keep("dk correction") * left * (U @ D.T) - keep("dk state") * y * (dV @ S.T) + keep("dk scores") * PO.T @ Q
                       + keep("dk keys") * PV.T @ K + keep("dk rows") * PV @ K)
        out[2][t:e], out[3][t:e] = dV, (X * E).sum(1)
        # by token: what reaches over its decay, from the tokens before it (and the state) to it and those behind (and D)
        F = keep("dld pairs") * (PO * (Q @ K.T) + PV * (K @ K.T))
        read = keep("dld read") * (y * (scale * (G * (Q @ S)) - dV * (K @ S))).sum(1)
        write = keep("dld write") * left[:, 0] * (U * (K @ D)).sum(1)
        for i in range(n):
            out[4][t + i] = F[i:, :i].sum() + read[i:].sum() + write[:i].sum() + keep("dld state") * y[-1, 0] * (D * S).sum()
        D = y[-1] * D + scale * (y * Q).T @ G - (y * K).T @ dV
    return (*out, D)


def turn(x, angles, interleaved=False, magnitude=1.0, inverse=False):
    """x (B, T, H, D), angles (B, T, pairs): the first 2 pairs coordinates turned."""
    n = angles.shape[-1]
    a = angles[:, :, None] * (-1.0 if inverse else 1.0)
    c, s = magnitude * np.cos(a), magnitude * np.sin(a)
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y = x.astype(float).copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def qk_norm(x, w=None, eps=1e-6, l2=False, angles=None, interleaved=False, magnitude=1.0):
    n = 1 if l2 else x.shape[-1]
    z = x / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)
    z = z if w is None else z * w
    return z if angles is None else turn(z, angles, interleaved, magnitude)


def qk_norm_backward(dy, x, w=None, eps=1e-6, l2=False, angles=None, interleaved=False, magnitude=1.0):
    """(dx, dw) of sum(dy * qk_norm(x))."""
    dz = dy if angles is None else turn(dy, angles, interleaved, magnitude, inverse=True)
    n = 1 if l2 else x.shape[-1]
    r = 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)
    t = dz if w is None else dz * w
    return r * t - x * r ** 3 * (t * x).sum(-1, keepdims=True) / n, (dz * x * r).sum((0, 1, 2))
