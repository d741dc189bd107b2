"""Pins of oracle/delta_oracle.py, each against something other than itself (CPU)."""

import numpy as np
import pytest
import torch

from oracle import delta_oracle as O
from oracle import layer_oracle as L


def _inputs(seed, T, dk, dv, unit=True):
    r = np.random.default_rng(seed)
    q, k = r.standard_normal((T, dk)), r.standard_normal((T, dk))
    if unit:
        k = k / np.linalg.norm(k, axis=1, keepdims=True)
    return (q, k, r.standard_normal((T, dv)), r.uniform(0, 1, T), -r.exponential(0.2, T), r.standard_normal((T, dv)),
            r.standard_normal((dk, dv)), r.standard_normal((dk, dv)))


@pytest.mark.parametrize("T", [1, 2, 17, 64, 65, 200])
def test_the_recurrence_is_the_chunked_closed_form(T):
    q, k, v, b, ld, _, S0, _ = _inputs(T, T, 6, 4)
    for s in (None, S0):
        for x, y in zip(O.delta_recurrent(q, k, v, b, ld, 0.3, s), O.delta_chunked(q, k, v, b, ld, 0.3, s)):
            np.testing.assert_allclose(x, y, rtol=1e-10, atol=1e-10)


def test_what_it_is_without_its_parts():
    q, k, v, b, ld, _, S0, _ = _inputs(3, 20, 5, 3)
    o, S = O.delta_recurrent(q, k, v, np.zeros(20), ld, 1.0, S0)           # nothing is written: the state fades
    np.testing.assert_allclose(S, np.exp(ld.sum()) * S0)
    np.testing.assert_allclose(o, np.exp(np.cumsum(ld))[:, None] * (q @ S0))
    e = np.eye(5)                                                         # orthogonal keys: nothing to correct
    o, S = O.delta_recurrent(q[:5], e, v[:5], np.ones(5), np.zeros(5))
    np.testing.assert_allclose(S, v[:5])
    o, S = O.delta_recurrent(q, k, v, np.ones(20), np.zeros(20), 1.0, S0)  # beta 1: the last value is read back
    np.testing.assert_allclose(k[-1] @ S, v[-1])
    o, S = O.delta_recurrent(q, k, v, b, np.full(20, -np.inf))             # no memory
    np.testing.assert_allclose(S, b[-1] * np.outer(k[-1], v[-1]))


def test_gradients_against_differences():
    q, k, v, b, ld, dO, S0, dS = _inputs(7, 6, 3, 4, unit=False)

    def loss(q, k, v, b, ld, S0):
        o, S = O.delta_recurrent(q, k, v, b, ld, 0.7, S0)
        return (dO * o).sum() + (dS * S).sum()

    got = O.delta_backward(q, k, v, b, ld, dO, 0.7, S0, dS)
    args, h = [q, k, v, b, ld, S0], 1e-6
    for i, g in enumerate(got):
        num = np.zeros_like(g)
        for at in np.ndindex(g.shape):
            lo, hi = [x.copy() for x in args], [x.copy() for x in args]
            lo[i][at] -= h
            hi[i][at] += h
            num[at] = (loss(*hi) - loss(*lo)) / (2 * h)
        # rounding of the differences, 1e-16 |loss| / h, and their third derivative, h^2 of it
        np.testing.assert_allclose(g, num, rtol=1e-6, atol=1e-6)


def test_gradients_against_autograd():
    arrays = _inputs(11, 90, 8, 6)
    q, k, v, b, ld, S0 = (torch.tensor(x, requires_grad=True) for x in (*arrays[:5], arrays[6]))
    dO, dS = torch.tensor(arrays[5]), torch.tensor(arrays[7])
    S, loss = S0, 0.0
    for t in range(90):
        S = torch.exp(ld[t]) * S
        S = S + torch.outer(k[t], b[t] * (v[t] - k[t] @ S))
        loss = loss + 0.4 * (q[t] @ S) @ dO[t]
    want = torch.autograd.grad(loss + (S * dS).sum(), (q, k, v, b, ld, S0))
    for g, w in zip(O.delta_backward(*arrays[:6], 0.4, arrays[6], arrays[7]), want):
        np.testing.assert_allclose(g, w.numpy(), rtol=1e-9, atol=1e-9)


def test_sizes_bound_what_they_are_sizes_of():
    q, k, v, b, ld, dO, S0, dS = _inputs(5, 150, 8, 6)
    _, S = O.delta_recurrent(q, k, v, b, ld, 1.0, S0)
    assert np.all(np.linalg.norm(S, axis=0) <= O.delta_sizes(q, k, v, b, ld, S0)[0])
    Bq, Bk, Bl = O.delta_gradient_sizes(q, k, v, b, ld, dO, 0.5, S0, dS)
    dq, dk, _, _, dl, _ = O.delta_backward(q, k, v, b, ld, dO, 0.5, S0, dS)
    for g, B in ((dq, Bq), (dk, Bk), (dl, Bl)):
        assert np.all(np.abs(g) <= B * (1 + 1e-9))


def test_turn_is_rotary():
    r = np.random.default_rng(1)
    x, pos, rates = r.standard_normal((2, 5, 3, 16)), r.integers(0, 99, (2, 5)), np.array([1.0, 0.3, 0.1])
    for il in (False, True):
        np.testing.assert_allclose(O.turn(x, pos[..., None] * rates, il, 1.5), L.rotary(x, pos, rates, il, 1.5))


@pytest.mark.parametrize("l2", [False, True])
def test_qk_norm_and_its_gradient(l2):
    r = np.random.default_rng(2)
    x, dy, w = r.standard_normal((2, 3, 2, 8)), r.standard_normal((2, 3, 2, 8)), r.standard_normal(8)
    angles = r.standard_normal((2, 3, 3))
    size = np.linalg.norm(O.qk_norm(x, eps=0.0, l2=l2), axis=-1)
    np.testing.assert_allclose(size, 1.0 if l2 else np.sqrt(8.0))
    f = lambda x, w: (dy * O.qk_norm(x, w, 1e-3, l2, angles, True, 1.2)).sum()  # noqa: E731
    dx, dw = O.qk_norm_backward(dy, x, w, 1e-3, l2, angles, True, 1.2)
    h = 1e-6
    for i, g in enumerate((dx, dw)):
        num = np.zeros_like(g)
        for at in np.ndindex(g.shape):
            lo, hi = [x.copy(), w.copy()], [x.copy(), w.copy()]
            lo[i][at] -= h
            hi[i][at] += h
            num[at] = (f(*hi) - f(*lo)) / (2 * h)
        np.testing.assert_allclose(g, num, rtol=1e-6, atol=1e-7)
