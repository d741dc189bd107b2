"""The gated delta rule on the GPU by the bounds of delta_norms.py: every output and gradient of every sequence and head, which a
wrong or missing term exceeds."""

import numpy as np
import pytest
import torch

import delta_norms as N
import kernelized_psd_feature_amd as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = N.BF, N.F32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def _run(args, scale=0.25, cu=None, forward=True):
    """The outputs and gradients by name of arguments as delta_norms.inputs returns them."""
    q, k, v, b, ld, dO, S0, dS = (None if x is None else x.to(DEV) for x in args)
    got = {}
    if forward:
        got["o"], got["state"] = K.fwd_delta(q, k, v, b, ld, scale=scale, initial_state=S0, return_state=True, cu_seqlens=cu)
        got["o alone"] = K.fwd_delta(q, k, v, b, ld, scale=scale, initial_state=S0, cu_seqlens=cu)
    grads = K.bwd_delta(q, k, v, b, dO, ld, scale=scale, initial_state=S0, dfinal_state=dS, cu_seqlens=cu)
    got.update((name, x) for name, x in zip(N.GRADIENTS, grads) if x is not None)
    return got


def _check(args, seqs, scale=0.25, cu=None, dtype=BF, forward=True):
    got = _run(args, scale, cu, forward)
    alone = got.pop("o alone", None)
    N.check(args, seqs, got, scale, dtype)
    if alone is not None:
        N.check(args, seqs, {"o": alone}, scale, dtype)
    return got


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("shape", N.SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_delta(dtype, shape, states):
    args = N.inputs(sum(shape), *shape, dtype)
    if not states:
        args[6:] = None, None
    _check(args, N.rows(*shape[:2]), dtype=dtype)


@pytest.mark.parametrize("shape", [(1, 1, 1, 2, 4, 4), (1, 70, 1, 2, 12, 20), (1, 300, 1, 2, 100, 68), (1, 130, 2, 2, 36, 124),
                                   (1, 200, 1, 3, 4, 128), (1, 130, 1, 2, 128, 4), (1, 90, 1, 1, 32, 92)])
def test_fp32_widths_of_odd_vectors(shape):
    args = N.inputs(sum(shape), *shape, F32)
    _check(args, N.rows(*shape[:2]), dtype=F32)


@pytest.mark.parametrize("lengths", N.PACKED)
@pytest.mark.parametrize("widths", [(64, 40), (32, 128), (128, 72)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_packed(dtype, widths, lengths):
    T = 3 + sum(lengths) + 70
    args = N.inputs(T, 1, T, 1, 2, *widths, dtype, n=len(lengths))
    cu = torch.tensor(3 + np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    _check(args, N.rows(1, T, lengths, 3), 0.5, cu, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_many_packed_sequences(dtype):
    # more sequences than a workgroup has threads, most of them of no or one token
    lengths = [(0, 1, 2, 0, 1, 70, 0, 3)[i * i % 8] for i in range(1500)]
    T = sum(lengths)
    args = N.inputs(5, 1, T, 1, 1, 16, 16, dtype, n=len(lengths))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    _check(args, N.rows(1, T, lengths), 0.5, cu, dtype)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0, "mixed"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_beta_over_its_range(dtype, beta, gated):
    args = N.inputs(8, 1, 260, 2, 2, 64, 64, dtype)
    if beta == "mixed":                              # tokens that write nothing or next to nothing among the others
        args[3][:, 50:90], args[3][:, 128], args[3][:, 130:140], args[3][:, 200:210] = 0.0, 0.0, 1e-12, 1e-20
    else:
        args[3].fill_(beta)
    if not gated:
        args[4] = None
    _check(args, N.rows(1, 260), 1.0, dtype=dtype)


@pytest.mark.parametrize("beta", [1.0, 2.0])
@pytest.mark.parametrize("shape", [(1, 200, 1, 1, 64, 64), (1, 200, 1, 2, 128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_keys_that_repeat(dtype, shape, beta):
    # one key over and over: the system is as far from the unit matrix as it gets
    args = N.inputs(12, *shape, dtype)
    args[1] = args[1][:, :1].expand_as(args[1]).contiguous()
    args[3].fill_(beta)
    args[4] = None
    _check(args, N.rows(*shape[:2]), 1.0, dtype=dtype)


@pytest.mark.parametrize("beta", [-1.5, 300.0, 3e4])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_steps_of_any_size(dtype, beta):
    # on keys short enough that the state stays bounded: beta k k^T is what beta in [0, 2] makes of unit keys
    args = N.inputs(61, 1, 200, 1, 2, 64, 40, dtype)
    args[1] = (args[1].float() * abs(beta) ** -0.5).to(dtype)
    args[2] = (args[2].float() * abs(beta) ** -0.5).to(dtype)
    args[3] = (args[3].float() * beta).to(dtype)
    if beta < 0:                                     # the state grows along a key: by a factor of 2.5 each time
        args[3][:, 10:] = 0.0
    _check(args, N.rows(1, 200), 1.0, dtype=dtype)


@pytest.mark.parametrize("ld", [-1.0, -5.0, -10.0, -20.0, -60.0])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_strong_decays(dtype, ld):
    # the gradient of a strong decay is small, e^ld of what its neighbours' terms are, and has to be as good as theirs
    for every in (1, 3):
        args = N.inputs(23, 1, 256, 1, 2, 64, 64, dtype)
        args[4][:, ::every] = ld * (0.5 + torch.rand(1, -(-256 // every), 2, generator=torch.Generator().manual_seed(1)))
        _check(args, N.rows(1, 256), 1.0, dtype=dtype)


@pytest.mark.parametrize("shape", [(1, 150, 2, 2, 64, 64), (1, 150, 1, 2, 128, 128), (2, 90, 1, 3, 32, 40)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_gradients_scale_with_what_arrives(dtype, shape):
    # linear in dO, down to 2^-66, about 1e-20, and where beta is zero, too.  A power of two changes no rounding; what it
    # takes below fp32's range is less than 2^-126 2^66 of what it is added to.  Two results are a step apart at most.
    args = N.inputs(31, *shape, dtype)
    args[3][:, 20:60:3], args[3][:, 64:70], args[3][:, 80] = 0.0, 1e-9, 1e-12
    args[7] = None
    whole = _run(args, forward=False)
    assert whole["db"][:, 20:60:3].any()
    for power in (-10, -30, -66):
        less = _run([*args[:5], (args[5].double() * 2.0 ** power).to(dtype), *args[6:]], forward=False)
        for name, x in whole.items():
            x = x.double()
            half = N.HALF[F32 if name in N.IN_FP32 else dtype]
            few = 2.0 ** -60 if power > -66 else 2.0 ** -24
            off = (less[name].double() * 2.0 ** -power - x).abs() - 2 * half * x.abs() - few * x.norm() / x.numel() ** 0.5
            assert off.max() <= 0, (name, power, float(off.max()))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_tokens_that_write_nothing_leave_no_gradient(dtype):
    # u is zero there: no gradient of v, and none of k but through the state that it would read and correct
    args = N.inputs(8, 1, 150, 2, 2, 64, 64, dtype)
    args[3].zero_()
    got = _run(args, forward=False)
    assert not got["dk"].any() and not got["dv"].any() and got["db"].any()


@pytest.mark.parametrize("at", [17, 41, 63])
def test_a_product_that_overflows_reaches_no_earlier_row(at):
    # k_at . k_5 = 1e23 and k_5 . k_3 = 1e16 are numbers, their product in the inverse is not; the rows before it are as without
    q, k, v, b, _, _, S0, _ = (x.to(DEV) for x in N.inputs(2, 1, 130, 1, 1, 64, 64, F32))
    k[0, 5] = k[0, 3]
    k[0, [3, 5]] *= 1e8
    clean, _ = K.fwd_delta(q, k, v, b, initial_state=S0, return_state=True)
    k[0, at] = k[0, 3] * 1e7
    o, S = K.fwd_delta(q, k, v, b, initial_state=S0, return_state=True)
    assert torch.isfinite(clean[:, :at]).all() and torch.equal(o[:, :at], clean[:, :at])
    assert not torch.isfinite(o[:, at:]).any() and not torch.isfinite(S).any()
