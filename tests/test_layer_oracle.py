"""Pins of oracle/layer_oracle.py, each against something other than itself (CPU)."""

import numpy as np
import pytest
import torch

from oracle import layer_oracle as L


def _inputs(seed, T, dk, dv):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, dk)), r.standard_normal((T, dk)), r.standard_normal((T, dv)),
            r.standard_normal((T, dv)), r.standard_normal((dk, dv)), r.standard_normal((dk, dv)))


@pytest.mark.parametrize("ld", [0.0, -0.01, -0.7, -50.0, -np.inf, 0.05])
@pytest.mark.parametrize("T", [1, 2, 17])
def test_decay_closed_form_is_the_recurrence(T, ld):
    q, k, v, _, S0, _ = _inputs(T, T, 5, 3)
    for s in (None, S0):
        o, S = L.decay_closed(q, k, v, ld, 0.3, s)
        ro, rS = L.decay_recurrent(q, k, v, ld, 0.3, s)
        np.testing.assert_allclose(o, ro, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(S, rS, rtol=1e-12, atol=1e-12)


def test_decay_of_one_is_a_running_sum_and_of_zero_the_token_itself():
    q, k, v, *_ = _inputs(3, 9, 4, 4)
    o, S = L.decay_closed(q, k, v, 0.0)
    np.testing.assert_allclose(S, k.T @ v)
    np.testing.assert_allclose(o[-1], q[-1] @ (k.T @ v))
    o, S = L.decay_closed(q, k, v, -np.inf)
    np.testing.assert_allclose(o, (q * k).sum(-1, keepdims=True) * v)
    np.testing.assert_allclose(S, np.outer(k[-1], v[-1]))


@pytest.mark.parametrize("ld", [0.0, -0.2])
def test_decay_backward_against_differences(ld):
    q, k, v, dO, S0, dS = _inputs(7, 6, 3, 4)

    def loss(q, k, v, S0):
        o, S = L.decay_closed(q, k, v, ld, 0.7, S0)
        return (dO * o).sum() + (dS * S).sum()

    got = L.decay_backward(q, k, v, dO, ld, 0.7, S0, dS)
    args = [q, k, v, S0]
    h = 1e-5
    for i, g in enumerate(got):
        num = np.zeros_like(g)
        for at in np.ndindex(g.shape):
            lo, hi = [x.copy() for x in args], [x.copy() for x in args]
            lo[i][at] -= h
            hi[i][at] += h
            num[at] = (loss(*hi) - loss(*lo)) / (2 * h)
        # the loss is a polynomial of degree 3: differences are off by rounding, 1e-16 |loss| / h
        np.testing.assert_allclose(g, num, atol=1e-8)


def test_decay_backward_against_autograd_of_the_recurrence():
    q, k, v, dO, S0, dS = _inputs(11, 40, 8, 6)
    leaves = [torch.tensor(x, requires_grad=True) for x in (q, k, v, S0)]
    tq, tk, tv, tS = leaves
    g, S, loss = float(np.exp(-0.1)), tS, 0.0
    for t in range(40):
        S = g * S + torch.outer(tk[t], tv[t])
        loss = loss + (torch.tensor(dO[t]) * (tq[t] @ S)).sum() * 0.5
    loss = loss + (S * torch.tensor(dS)).sum()
    want = torch.autograd.grad(loss, leaves)
    for g_, w_ in zip(L.decay_backward(q, k, v, dO, -0.1, 0.5, S0, dS), want):
        np.testing.assert_allclose(g_, w_.numpy(), rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_complex_product_and_inverts(interleaved):
    r = np.random.default_rng(5)
    x = r.standard_normal((2, 3, 2, 10))
    pos = np.array([[0, 1, 2], [100000, 7, 3]])
    rates = np.array([1.0, 0.1, 0.003])
    y = L.rotary(x, pos, rates, interleaved, 1.0)
    a, b = (x[..., 0:6:2], x[..., 1:6:2]) if interleaved else (x[..., :3], x[..., 3:6])
    z = (a + 1j * b) * np.exp(1j * pos[..., None, None] * rates)
    ya, yb = (y[..., 0:6:2], y[..., 1:6:2]) if interleaved else (y[..., :3], y[..., 3:6])
    np.testing.assert_allclose(ya, z.real, atol=1e-12)
    np.testing.assert_allclose(yb, z.imag, atol=1e-12)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    np.testing.assert_allclose(L.rotary(y, pos, rates, interleaved, 1.0, True), x, atol=1e-12)
    np.testing.assert_allclose(y[0, 0], x[0, 0], atol=0)         # position 0


def test_rotary_scores_depend_on_the_distance_alone():
    r = np.random.default_rng(6)
    q, k = r.standard_normal((2, 1, 1, 1, 8))
    rates = 10000.0 ** (-np.arange(4) / 4)
    at = lambda x, p: L.rotary(x, np.array([[p]]), rates)[0, 0, 0]  # noqa: E731
    want = at(q, 5) @ at(k, 2)
    for shift in (1, 1000, 12345):
        np.testing.assert_allclose(at(q, 5 + shift) @ at(k, 2 + shift), want, atol=1e-9)


def test_layer_norm_rows_and_gradients():
    r = np.random.default_rng(8)
    x, w, b, dy = r.standard_normal((4, 7)), r.standard_normal(7), r.standard_normal(7), r.standard_normal((4, 7))
    y, mean, rstd = L.layer_norm(x, w, b, 1e-3)
    want = torch.nn.functional.layer_norm(*(torch.tensor(t) for t in (x,)), (7,), torch.tensor(w), torch.tensor(b), 1e-3)
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-12, atol=1e-12)
    got = L.layer_norm_backward(dy, x, w, 1e-3)
    h = 1e-6
    f = lambda x, w, b: (dy * L.layer_norm(x, w, b, 1e-3)[0]).sum()  # noqa: E731
    for i, g in enumerate(got):
        args, num = [x, w, b], np.zeros_like(g)
        for at in np.ndindex(g.shape):
            lo, hi = [t.copy() for t in args], [t.copy() for t in args]
            lo[i][at] -= h
            hi[i][at] += h
            num[at] = (f(*hi) - f(*lo)) / (2 * h)
        np.testing.assert_allclose(g, num, atol=1e-7)
