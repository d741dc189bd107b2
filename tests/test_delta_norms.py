"""The bounds of delta_norms.py without a GPU: they hold for the formulas in 64 bits, and for each shape that a GPU test uses
they reject zeros and every gradient that lacks a term of its formula."""

import functools

import numpy as np
import pytest
import torch

import delta_norms as N
from oracle import delta_oracle as O

TERMS = {"dq": ("state", "pairs"), "dk": ("correction", "state", "scores", "keys", "rows"),
         "dld": ("state", "read", "write", "pairs"), "db": ("inverse",)}


def _differs(x, y):
    return np.linalg.norm(x - y) > 1e-9 * np.linalg.norm(y)


@pytest.mark.parametrize("dtype", [N.BF, N.F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", N.SHAPES)
def test_the_bounds_reject_gradients_without_a_term(shape, dtype):
    args = N.inputs(sum(shape), *shape, dtype)
    seqs = N.rows(*shape[:2])
    want = N.expected(args, seqs, 0.25, forward=False)
    for key, (x, size) in N.expected(args, seqs, 0.25, backward=O.delta_chunked_backward, forward=False).items():
        assert N.share_of_bound(x, want[key][0], size, key[0], dtype) < 1e-3, key
    for key, (ref, size) in want.items():
        assert not N.share_of_bound(0.0 * ref, ref, size, key[0], dtype) <= 4.0, key
        assert not N.share_of_bound(np.nan * ref, ref, size, key[0], dtype) <= 1.0
    for name, terms in TERMS.items():
        for term in terms:
            lacking = N.expected(args, seqs, 0.25, forward=False, sizes=lambda *a: dict.fromkeys(N.GRADIENTS, 0.0),
                                 backward=functools.partial(O.delta_chunked_backward, without=f"{name} {term}"))
            differ = [k for k, x in lacking.items() if k[0] == name and _differs(x[0], want[k][0])]
            assert differ or shape[1] == 1, (name, term)   # a single token has no pairs
            # (of a few tokens a head may hardly have the term)
            shares = [N.share_of_bound(lacking[k][0], *want[k], name, dtype) for k in differ]
            assert not shares or max(shares) > 1.0, (name, term, shares)


@pytest.mark.parametrize("lengths", N.PACKED)
def test_the_bounds_reject_zeros_of_packed_sequences(lengths):
    T = 3 + sum(lengths) + 70
    args = N.inputs(T, 1, T, 1, 2, 64, 40, N.BF, n=len(lengths))
    for key, (ref, size) in N.expected(args, N.rows(1, T, lengths, 3), 0.5).items():
        if ref.size and np.any(ref):
            assert not N.share_of_bound(0.0 * ref, ref, size, key[0], N.BF) <= 4.0, key


def test_rows_and_heads_are_those_of_the_arguments():
    lengths = [2, 0, 3]
    args = N.inputs(1, 1, 9, 1, 2, 8, 8, N.F32, n=3)
    seqs = N.rows(1, 9, lengths, 1)
    assert seqs == [(0, 1, 2), (0, 3, 0), (0, 3, 3)]
    got = N.results(args, seqs, {"dv": args[2], "dS0": args[6]})
    assert np.array_equal(got["dv", 2, 1], args[2][0, 3:6, 1].double().numpy())
    assert np.array_equal(got["dS0", 1, 0], args[6][1, 0].double().numpy())
    for i, h, hk, b, s, a in N.heads(args, seqs, 1.0):
        assert hk == 0 and np.array_equal(a[3], args[3][0, s, h].double().numpy()) and np.array_equal(a[7], args[6][i, h].double().numpy())
    assert torch.equal(args[0], N.inputs(1, 1, 9, 1, 2, 8, 8, N.F32, n=3)[0])
