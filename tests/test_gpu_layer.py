"""Decayed linear attention, rotary positions and layer norm on the GPU against the fp64 oracle.

Tolerances are bounds, taken elementwise from sums of absolute terms.  A rounding to bf16 is off by
at most 2^-8 of the value, one to fp32 by 2^-24.
  attention: an output is a sum of terms with the absolute sum B.  bf16 rounds a term's factors at
    most twice (the weight of a pair; or the term's share of the state as it is added and as it is
    read), and the result once: 2 2^-8 B + 2^-8 |o|.  In fp32 a term passes at most 2 T + dk + 64
    additions and products, and T / 64 + 4 powers of the decay, good to 2^-21 each.  A state that is
    returned is rounded in fp32 only.
  rotary: an angle is reduced in fp64 and rounded to 2^-24 of half a turn, the sine and cosine are good to
    2^-23, so is each product: together below 2^-21 (|a| + |b|) m, and the result's rounding.
  layer norm: a row's sums run over at most c = 64 + N / 256 additions a lane and tree (N below 64):
    the mean is off by c 2^-24 of the mean |x|, which moves every normalized value.
"""

import numpy as np
import pytest
import torch

import kernelized_psd_feature_amd as K
from kernelized_psd_feature_amd import layer as KL
from oracle import layer_oracle as L

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def _np(x):
    return x.detach().to(torch.float64).cpu().numpy()


def _randn(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def _inside(got, ref, tol, what):
    g = _np(got)
    bad = ~(np.abs(g - ref) <= tol + 1e-30)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(g - ref) - tol, -1.0)), g.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {g.size} off, worst at {at}: {g[at]} for {ref[at]}, "
                             f"tolerance {np.broadcast_to(tol, g.shape)[at]}")
    print(f"{what}: worst share of the tolerance {np.max(np.abs(g - ref) / (tol + 1e-30)):.3f}", flush=True)


def _decay_tol(ref, size, T, dk, dtype, state=False):
    few = (2 * T + dk + 64) * 2.0 ** -24 + (T / 64 + 4) * 2.0 ** -21
    if state or dtype == F32:
        return (few + 2.0 ** -22) * size + 2.0 ** -24 * np.abs(ref)
    return (2 * U[BF] * 1.02 + few) * size + U[BF] * 1.01 * np.abs(ref)


def _decays(H, kind="mixed"):
    if kind == "mixed":
        return torch.log1p(-(2.0 ** -(1 + 8 * torch.arange(H, dtype=torch.float64) / max(1, H - 1)))).float().to(DEV)
    return torch.full((H,), float(kind), device=DEV)


def _sequences(B, T, lengths):
    if lengths is None:
        return [(b, 0, T) for b in range(B)]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    return [(0, int(cu[i]), int(n)) for i, n in enumerate(lengths)]


def _check_decay(q, k, v, ld, scale, lengths=None, S0=None, dO=None, dS=None, o=None, S=None, grads=None,
                 what=""):
    """Outputs, final states and gradients of every sequence and head against the oracle."""
    B, T, H, dk = q.shape
    nq, nk, nv, nld = _np(q), _np(k), _np(v), _np(ld)
    for n, (b, t0, len_) in enumerate(_sequences(B, T, lengths)):
        rows = slice(t0, t0 + len_)
        for h in range(H):
            a = [x[b, rows, h] for x in (nq, nk, nv)]
            s0 = None if S0 is None else _np(S0)[n, h]
            ab = [np.abs(x) for x in a]
            s0b = None if s0 is None else np.abs(s0)
            ro, rS = L.decay_closed(*a, nld[h], scale, s0)
            bo, bS = L.decay_closed(*ab, nld[h], abs(scale), s0b)
            tag = f"{what} seq {n} (len {len_}) head {h}"
            if o is not None and len_:
                _inside(o[b, rows, h], ro, _decay_tol(ro, bo, len_, dk, q.dtype), tag + " o")
            if S is not None:
                _inside(S[n, h], rS, _decay_tol(rS, bS, len_, dk, q.dtype, True), tag + " state")
            if grads is not None:
                g = _np(dO)[b, rows, h]
                ds = None if dS is None else _np(dS)[n, h]
                refs = L.decay_backward(*a, g, nld[h], scale, s0, ds)
                sizes = L.decay_backward(*ab, np.abs(g), nld[h], abs(scale), s0b, None if ds is None else np.abs(ds))
                for name, got, r, z in zip(("dq", "dk", "dv"), grads, refs, sizes):
                    if len_:
                        _inside(got[b, rows, h], r, _decay_tol(r, z, len_, 128, q.dtype), f"{tag} {name}")
                if grads[3] is not None:
                    _inside(grads[3][n, h], refs[3], _decay_tol(refs[3], sizes[3], len_, 128, q.dtype, True),
                            tag + " dS0")


# ---- decayed linear attention ------------------------------------------------------------------

# lengths around the chunk of 64, long enough for several segments, all widths of the tiles
SHAPES = [(1, 1, 1, 64, 64), (2, 2, 3, 64, 64), (1, 63, 2, 64, 64), (1, 64, 2, 64, 64), (1, 65, 2, 64, 64),
          (2, 129, 2, 32, 64), (1, 1000, 2, 64, 64), (1, 700, 1, 128, 128), (1, 330, 3, 40, 72),
          (3, 200, 1, 16, 128), (1, 577, 2, 128, 24), (1, 260, 2, 104, 8), (2, 70, 2, 8, 8), (1, 321, 1, 96, 64)]


@pytest.mark.parametrize("initial", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_forward_and_state(dtype, shape, initial):
    B, T, H, dk, dv = shape
    print("case", dtype, shape, initial, flush=True)
    q, k, v = _randn(1, B, T, H, dk, dtype=dtype), _randn(2, B, T, H, dk, dtype=dtype), _randn(3, B, T, H, dv, dtype=dtype)
    S0 = _randn(4, B, H, dk, dv) if initial else None
    ld = _decays(H)
    o, S = K.fwd_decay(q, k, v, ld, scale=0.25, initial_state=S0, return_state=True)
    assert o.dtype == dtype and S.dtype == F32
    _check_decay(q, k, v, ld, 0.25, S0=S0, o=o, S=S)
    o2 = K.fwd_decay(q, k, v, ld, scale=0.25, initial_state=S0)
    _check_decay(q, k, v, ld, 0.25, S0=S0, o=o2, what="no state")
    again, _ = K.fwd_decay(q, k, v, ld, scale=0.25, initial_state=S0, return_state=True)
    assert torch.equal(o, again)


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_backward(dtype, shape, states):
    B, T, H, dk, dv = shape
    print("case", dtype, shape, states, flush=True)
    q, k, v, g = (_randn(i, B, T, H, d, dtype=dtype) for i, d in ((5, dk), (6, dk), (7, dv), (8, dv)))
    S0, dS = (_randn(9, B, H, dk, dv), _randn(10, B, H, dk, dv)) if states else (None, None)
    ld = _decays(H)
    grads = K.bwd_decay(q, k, v, g, ld, scale=0.5, initial_state=S0, dfinal_state=dS)
    assert (grads[3] is not None) == states
    _check_decay(q, k, v, ld, 0.5, S0=S0, dO=g, dS=dS, grads=grads)
    again = K.bwd_decay(q, k, v, g, ld, scale=0.5, initial_state=S0, dfinal_state=dS)
    assert all(x is y or torch.equal(x, y) for x, y in zip(grads, again))


@pytest.mark.parametrize("T,dk,dv", [(1, 4, 4), (70, 12, 20), (300, 100, 68), (513, 36, 124), (700, 4, 128), (260, 128, 4)])
def test_decay_fp32_widths_of_odd_vectors(T, dk, dv):
    # rows of four fp32 elements and odd multiples of it, which bf16 does not have
    B, H = 2, 2
    q, k, v, g = (_randn(i, B, T, H, d) for i, d in ((1, dk), (2, dk), (3, dv), (4, dv)))
    S0, dS, ld = _randn(5, B, H, dk, dv), _randn(6, B, H, dk, dv), _decays(H)
    o, S = K.fwd_decay(q, k, v, ld, initial_state=S0, return_state=True)
    grads = K.bwd_decay(q, k, v, g, ld, initial_state=S0, dfinal_state=dS)
    _check_decay(q, k, v, ld, 1.0, S0=S0, dO=g, dS=dS, o=o, S=S, grads=grads)
    st = S0.clone()
    _check_decay(q, k, v, ld, 1.0, S0=S0, o=K.decode_decay(q, k, v, ld, st), S=st)


@pytest.mark.parametrize("ld", ["0.0", "-1e-4", "-3.0", "-40.0", "-inf", "0.02"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_of_any_strength(dtype, ld):
    q, k, v, g = (_randn(i, 1, 300, 2, 64, dtype=dtype) for i in range(4))
    S0, dS = _randn(5, 1, 2, 64, 64), _randn(6, 1, 2, 64, 64)
    decays = _decays(2, ld)
    o, S = K.fwd_decay(q, k, v, decays, initial_state=S0, return_state=True)
    grads = K.bwd_decay(q, k, v, g, decays, initial_state=S0, dfinal_state=dS)
    _check_decay(q, k, v, decays, 1.0, S0=S0, dO=g, dS=dS, o=o, S=S, grads=grads)


@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 3, 8, 64])
def test_decay_of_few_tokens_keeps_its_weights(T, dk, dv):
    """One chunk without an entry state: a weight's two bf16 terms leave 2^-16 of it, so the outputs and
    gradients are off by little more than their own rounding."""
    B, H, scale = 2, 3, dk ** -0.5
    q, k = _randn(1, B, T, H, dk, dtype=BF), _randn(2, B, T, H, dk, dtype=BF)
    v, dO = _randn(3, B, T, H, dv, dtype=BF), _randn(4, B, T, H, dv, dtype=BF)
    ld = _decays(H)
    o = K.fwd_decay(q, k, v, ld, scale=scale)
    grads = K.bwd_decay(q, k, v, dO, ld, scale=scale)
    few = (2 * T + 128 + 64) * 2.0 ** -24 + 5 * 2.0 ** -21 + 1.02 * 2.0 ** -16
    for b in range(B):
        for h in range(H):
            a, g = [_np(x)[b, :, h] for x in (q, k, v)], _np(dO)[b, :, h]
            ab = [np.abs(x) for x in a]
            nld = _np(ld)[h]
            refs = (L.decay_closed(*a, nld, scale, None)[0], *L.decay_backward(*a, g, nld, scale, None, None)[:3])
            sizes = (L.decay_closed(*ab, nld, scale, None)[0],
                     *L.decay_backward(*ab, np.abs(g), nld, scale, None, None)[:3])
            for name, got, r, z in zip(("o", "dq", "dk", "dv"), (o, *grads), refs, sizes):
                _inside(got[b, :, h], r, few * z + U[BF] * 1.01 * np.abs(r), f"{name} batch {b} head {h}")


@pytest.mark.parametrize("T", [600, 2000])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128)])
def test_decay_first_rows_of_a_long_prompt_keep_their_weights(T, dk, dv):
    """The first chunk of a sequence has few weights a row and no entry state, however long the sequence
    is: the same bound as of a call with these rows alone."""
    H, n, scale = 3, 64, dk ** -0.5
    q, k, v = (_randn(i, 1, T, H, d, dtype=BF) for i, d in ((1, dk), (2, dk), (3, dv)))
    dO, ld = _randn(4, 1, T, H, dv, dtype=BF), _decays(H)
    o = K.fwd_decay(q, k, v, ld, scale=scale)
    _, gk, gv, _ = K.bwd_decay(q, k, v, dO, ld, scale=scale)
    few = (2 * n + 128 + 64) * 2.0 ** -24 + 5 * 2.0 ** -21 + 1.02 * 2.0 ** -16
    for h in range(H):
        nld = _np(ld)[h]
        a = [_np(x)[0, :n, h] for x in (q, k, v)]
        r, z = L.decay_closed(*a, nld, scale)[0], L.decay_closed(*[np.abs(x) for x in a], nld, scale)[0]
        _inside(o[0, :n, h], r, few * z + U[BF] * 1.01 * np.abs(r), f"o head {h}")
        # the gradients of keys and values run from the last token back: its last 64 rows
        a, g = [_np(x)[0, T - n:, h] for x in (q, k, v)], _np(dO)[0, T - n:, h]
        refs = L.decay_backward(*a, g, nld, scale)
        sizes = L.decay_backward(*[np.abs(x) for x in a], np.abs(g), nld, scale)
        for name, got, i in (("dk", gk, 1), ("dv", gv, 2)):
            _inside(got[0, T - n:, h], refs[i], few * sizes[i] + U[BF] * 1.01 * np.abs(refs[i]), f"{name} head {h}")


@pytest.mark.parametrize("ld", ["-inf", "-40.0", "-20.0"])
@pytest.mark.parametrize("T", [513, 700, 2000])
def test_decay_that_leaves_one_weight_keeps_it(T, ld):
    """g <= 2^-28: a row is its own pair, wherever it stands; what is left of the other tokens is below
    2^-28 of the absolute sums, whatever their rounding."""
    q, k, v, dO = (_randn(i, 1, T, 2, 64, dtype=BF) for i in range(4))
    decays = _decays(2, ld)
    o = K.fwd_decay(q, k, v, decays, scale=0.125)
    grads = K.bwd_decay(q, k, v, dO, decays, scale=0.125)
    few = (2 * 64 + 128 + 64) * 2.0 ** -24 + 5 * 2.0 ** -21 + 1.02 * 2.0 ** -16
    for h in range(2):
        a, g, nld = [_np(x)[0, :, h] for x in (q, k, v)], _np(dO)[0, :, h], _np(decays)[h]
        ab = [np.abs(x) for x in a]
        refs = (L.decay_closed(*a, nld, 0.125)[0], *L.decay_backward(*a, g, nld, 0.125)[:3])
        sizes = (L.decay_closed(*ab, nld, 0.125)[0], *L.decay_backward(*ab, np.abs(g), nld, 0.125)[:3])
        for name, got, r, z in zip(("o", "dq", "dk", "dv"), (o, *grads), refs, sizes):
            _inside(got[0, :, h], r, few * z + U[BF] * 1.01 * np.abs(r), f"{name} head {h}")


def _operands_rounded(a, b, c, ld, E):
    """One head's recurrence in fp64 (its own time order, entry state E) with the roundings to bf16 that
    the kernel's comments name, and no others: an output, the entry state of a chunk as it is read, and
    a pair's weight behind the first 512 rows of a head whose rows have four weights and more in effect."""
    bf = lambda x: torch.from_numpy(x).to(BF).double().numpy()  # noqa: E731
    out = np.zeros((a.shape[0], c.shape[1]))
    for at in range(0, a.shape[0], 64):
        A, B, C = (x[at:at + 64] for x in (a, b, c))
        n = A.shape[0]
        w = L.decay_weights(ld, n) * (A @ B.T)
        if at >= 512 and np.exp(2 * ld) >= 0.75:
            w = bf(w)
        out[at:at + 64] = w @ C + np.exp(ld * np.arange(n))[:, None] * (A @ bf(E))
        E = np.exp(ld * n) * E + (B * np.exp(ld * (n - np.arange(n)))[:, None]).T @ C
    return bf(out)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (40, 72)])
@pytest.mark.parametrize("T", [65, 300, 512, 513, 2000])
def test_decay_rounds_what_it_says_and_no_more(T, dk, dv):
    """The error's norm against that of the same roundings in fp64.  The scale is a power of two, so the
    same values are rounded (but those that fp32 sums put on the other side of a border, some 2^-12 of
    them), and the two norms agree to well within a percent.  With the terms taken out of this model, one
    less of the state's update makes the error 1.16 times as large and more where the state decays
    slowly (from 300 tokens on), one less of the weights 1.2 to 1.5 times where they are few."""
    scale = 0.125
    ld = torch.tensor([-0.002, -0.02, -0.1, -1.0], device=DEV)
    H = ld.numel()
    q, k = _randn(1, 1, T, H, dk, dtype=BF), _randn(2, 1, T, H, dk, dtype=BF)
    v, dO = _randn(3, 1, T, H, dv, dtype=BF), _randn(4, 1, T, H, dv, dtype=BF)
    S0, dS = _randn(5, 1, H, dk, dv), _randn(6, 1, H, dk, dv)
    o = K.fwd_decay(q, k, v, ld, scale=scale, initial_state=S0)
    grads = K.bwd_decay(q, k, v, dO, ld, scale=scale, initial_state=S0, dfinal_state=dS)
    for h in range(H):
        (a, b, c), g, nld = [_np(x)[0, :, h] for x in (q, k, v)], _np(dO)[0, :, h], _np(ld)[h]
        s0, ds = _np(S0)[0, h], _np(dS)[0, h]
        exact = (L.decay_closed(a, b, c, nld, scale, s0)[0], *L.decay_backward(a, b, c, g, nld, scale, s0, ds)[:3])
        a, b, c, g = (x[::-1] for x in (a, b, c, g))
        model = (_operands_rounded(scale * a[::-1], b[::-1], c[::-1], nld, np.exp(nld) * s0),
                 _operands_rounded(scale * g[::-1], c[::-1], b[::-1], nld, np.exp(nld) * s0.T),
                 _operands_rounded(c, scale * g, a, nld, ds.T)[::-1],
                 _operands_rounded(b, scale * a, g, nld, ds)[::-1])
        for name, got, m, r in zip(("o", "dq", "dk", "dv"), (o, *grads), model, exact):
            e, em = (np.linalg.norm(x - r) / np.linalg.norm(r) for x in (_np(got)[0, :, h], m))
            print(f"T {T} head {h} {name}: error {e:.6f}, of the roundings {em:.6f}", flush=True)
            assert e <= 1.03 * em, (name, h, e, em)


@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 5, 0], [64, 64, 64], [1, 0, 77, 512, 130, 1, 63],
                                     [700, 3], [5] * 30, [256, 1, 255, 257]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_packed(dtype, lengths):
    T, H, dk, dv = sum(lengths) + 13, 2, 64, 40      # 13 rows behind the last sequence
    print("case", dtype, lengths, flush=True)
    q, k, v, g = (_randn(i, 1, T, H, d, dtype=dtype) for i, d in ((1, dk), (2, dk), (3, dv), (4, dv)))
    n = len(lengths)
    S0, dS = _randn(5, n, H, dk, dv), _randn(6, n, H, dk, dv)
    ld = _decays(H)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    o, S = K.fwd_decay(q, k, v, ld, initial_state=S0, return_state=True, cu_seqlens=cu)
    grads = K.bwd_decay(q, k, v, g, ld, initial_state=S0, dfinal_state=dS, cu_seqlens=cu)
    _check_decay(q, k, v, ld, 1.0, lengths, S0=S0, dO=g, dS=dS, o=o, S=S, grads=grads)
    # rows behind the last sequence: zero in a new output, untouched in the caller's
    end = T - 13
    for x in (o, *grads[:3]):
        assert not x[:, end:].any()
    mine = torch.full_like(v, 7.0)
    K.fwd_decay(q, k, v, ld, initial_state=S0, cu_seqlens=cu, out=mine)
    assert (mine[:, end:] == 7.0).all()
    o2 = K.fwd_decay(q, k, v, ld, initial_state=S0, cu_seqlens=cu)
    assert torch.equal(mine[:, :end], o2[:, :end])
    # rows behind hold anything: they reach nothing
    for x in (q, k, v, g):
        x[:, end:] = float("nan")
    o3, S3 = K.fwd_decay(q, k, v, ld, initial_state=S0, return_state=True, cu_seqlens=cu)
    assert torch.equal(o3, o) and torch.equal(S3, S)
    again = K.bwd_decay(q, k, v, g, ld, initial_state=S0, dfinal_state=dS, cu_seqlens=cu)
    assert all(torch.equal(x, y) for x, y in zip(grads, again))


def test_decay_packed_offsets_outside_the_rows_are_clamped():
    q, k, v = (_randn(i, 1, 100, 2, 64, dtype=BF) for i in range(3))
    ld = _decays(2)
    o = K.fwd_decay(q, k, v, ld, cu_seqlens=torch.tensor([-5, 40, 1 << 30], dtype=torch.int32, device=DEV))
    _check_decay(q, k, v, ld, 1.0, [40, 60], o=o)


def test_decay_packed_first_rows_before_the_first_sequence_are_left_alone():
    q, k, v = (_randn(i, 1, 100, 1, 64, dtype=BF) for i in range(3))
    out = torch.full_like(v, 3.0)
    K.fwd_decay(q, k, v, _decays(1), cu_seqlens=torch.tensor([10, 80], dtype=torch.int32, device=DEV), out=out)
    assert (out[:, :10] == 3.0).all() and (out[:, 80:] == 3.0).all()
    _check_decay(q[:, 10:80], k[:, 10:80], v[:, 10:80], _decays(1), 1.0, o=out[:, 10:80])
    for cu in ([10, 80], [10, 10, 80], [100, 100], [64, 70]):        # and zero in a new output
        new = K.fwd_decay(q, k, v, _decays(1), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        assert not new[:, :cu[0]].any() and not new[:, cu[-1]:].any()
    out[:, :10], out[:, 80:] = 0, 0
    new = K.fwd_decay(q, k, v, _decays(1), cu_seqlens=torch.tensor([10, 10, 80], dtype=torch.int32, device=DEV))
    assert torch.equal(new, out)                     # an empty sequence in front changes nothing


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_strides(dtype):
    B, T, H, d = 2, 150, 4, 64
    ld = _decays(H)
    fused = _randn(1, B, T, H, 3 * d, dtype=dtype)   # q, k, v side by side
    q, k, v = fused.split(d, dim=-1)
    g = _randn(2, B, H, T, d, dtype=dtype).transpose(1, 2)      # head-major
    want = K.fwd_decay(q.contiguous(), k.contiguous(), v.contiguous(), ld)
    out = torch.empty(B, H, T, d, dtype=dtype, device=DEV).transpose(1, 2)
    assert K.fwd_decay(q, k, v, ld, out=out) is out and torch.equal(out, want)
    a = K.bwd_decay(q, k, v, g, ld)
    b = K.bwd_decay(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), ld)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    # heads that share their keys, a batch that shares its values
    ks, vs = k[:, :, :1].expand(B, T, H, d), v[:1].expand(B, T, H, d)
    want = K.fwd_decay(q, ks.contiguous(), vs.contiguous(), ld)
    assert torch.equal(K.fwd_decay(q, ks, vs, ld), want)
    st = _randn(3, B, H, d, d)
    s1, s2 = st.clone(), st.clone()
    assert torch.equal(K.decode_decay(q, ks, vs, ld, s1), K.decode_decay(q, ks.contiguous(), vs.contiguous(), ld, s2))
    assert torch.equal(s1, s2)


@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("shape", [(1, 1, 64, 64), (3, 4, 64, 64), (2, 3, 128, 128), (2, 2, 40, 72), (1, 2, 8, 8),
                                   (5, 1, 104, 24)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_decode(dtype, shape, T):
    B, H, dk, dv = shape
    q, k, v = (_randn(i, B, T, H, d, dtype=dtype) for i, d in ((1, dk), (2, dk), (3, dv)))
    st = _randn(4, B, H, dk, dv)
    S0, ld = st.clone(), _decays(H)
    o = K.decode_decay(q, k, v, ld, st, scale=0.5)
    nq, nk, nv, nld, ns = _np(q), _np(k), _np(v), _np(ld), _np(S0)
    for b in range(B):
        for h in range(H):
            a = [x[b, :, h] for x in (nq, nk, nv)]
            ro, rS = L.decay_recurrent(*a, nld[h], 0.5, ns[b, h])
            bo, bS = L.decay_closed(*[np.abs(x) for x in a], nld[h], 0.5, np.abs(ns[b, h]))
            few = (2 * T + dk + 16) * 2.0 ** -23     # fp32 throughout, the output rounded once
            _inside(o[b, :, h], ro, few * bo + U[dtype] * 1.01 * np.abs(ro), f"o {b} {h}")
            _inside(st[b, h], rS, few * bS, f"state {b} {h}")


@pytest.mark.parametrize("B,H,dk,dv", [(65536, 1, 16, 16), (70001, 2, 16, 24)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_decode_of_more_sequences_than_a_grid_axis_has(dtype, B, H, dk, dv):
    q, k, v = (_randn(i, B, 1, H, d, dtype=dtype) for i, d in ((1, dk), (2, dk), (3, dv)))
    st, ld = _randn(4, B, H, dk, dv), _decays(H)
    parts = [(slice(0, 40000), st[:40000].clone()), (slice(40000, B), st[40000:].clone())]
    S0 = st.clone()
    o = K.decode_decay(q, k, v, ld, st, scale=0.5)
    for rows, s in parts:
        assert torch.equal(o[rows], K.decode_decay(q[rows], k[rows], v[rows], ld, s, scale=0.5))
        assert torch.equal(st[rows], s)
    for b in (0, 65534, 65535, B - 1):
        for h in range(H):
            a = [_np(x[b, :, h]) for x in (q, k, v)]
            ro, rS = L.decay_recurrent(*a, _np(ld)[h], 0.5, _np(S0[b, h]))
            bo, bS = L.decay_closed(*[np.abs(x) for x in a], _np(ld)[h], 0.5, np.abs(_np(S0[b, h])))
            few = (2 + dk + 16) * 2.0 ** -23         # as in test_decay_decode
            _inside(o[b, :, h], ro, few * bo + U[dtype] * 1.01 * np.abs(ro), f"o {b} {h}")
            _inside(st[b, h], rS, few * bS, f"state {b} {h}")


def test_decay_decode_with_decays_zero_and_one():
    q, k, v = (_randn(i, 2, 3, 2, 64) for i in range(3))
    st = _randn(4, 2, 2, 64, 64)
    ld = torch.tensor([0.0, float("-inf")], device=DEV)
    S0 = st.clone()
    o = K.decode_decay(q, k, v, ld, st)
    _check_decay(q, k, v, ld, 1.0, S0=S0, o=o, S=st)


@pytest.mark.parametrize("at", [0, 17, 63, 64, 100, 255, 299])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_non_finite_tokens_reach_no_earlier_row(dtype, value, at):
    T = 300
    q, k, v, g = (_randn(i, 1, T, 1, 64, dtype=dtype) for i in range(4))
    ld = _decays(1, "-0.05")
    clean = K.fwd_decay(q, k, v, ld)
    # a value: only its own column, from its row on
    bad = v.clone()
    bad[0, at, 0, 21] = value
    o = K.fwd_decay(q, k, bad, ld)
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[0, at:, 0, 21] = False
    assert torch.isfinite(o[keep]).all() and not torch.isfinite(o[~keep]).any()
    fixed = torch.where(keep, o, clean)              # the rest agrees with the oracle on clean inputs
    _check_decay(q, k, v, ld, 1.0, o=fixed)
    # a key: every row from its own on, earlier rows bit for bit
    bad = k.clone()
    bad[0, at, 0, 5] = value
    o = K.fwd_decay(q, bad, v, ld)
    assert torch.equal(o[:, :at], clean[:, :at]) and not torch.isfinite(o[:, at:]).all(-1).any()
    # a query: its own row alone
    bad = q.clone()
    bad[0, at, 0, 5] = value
    o = K.fwd_decay(bad, k, v, ld)
    rest = [t for t in range(T) if t != at]
    assert torch.equal(o[:, rest], clean[:, rest]) and not torch.isfinite(o[:, at]).any()
    # the gradient of a row reaches the keys and values up to it
    ref = K.bwd_decay(q, k, v, g, ld)
    bad = g.clone()
    bad[0, at, 0, 33] = value
    dq, dk, dv, _ = K.bwd_decay(q, k, v, bad, ld)
    assert torch.equal(dq[:, rest], ref[0][:, rest])
    assert torch.equal(dk[:, at + 1:], ref[1][:, at + 1:])
    assert torch.isfinite(dv[:, at + 1:]).all() and not torch.isfinite(dv[0, :at + 1, 0, 33]).any()


def test_decay_empty_tensors():
    ld = _decays(2)
    S0 = _randn(1, 3, 2, 64, 64)
    q = torch.empty(3, 0, 2, 64, device=DEV, dtype=BF)
    o, S = K.fwd_decay(q, q, q, ld, initial_state=S0, return_state=True)
    assert o.shape == q.shape and torch.equal(S, S0)
    o, S = K.fwd_decay(q, q, q, ld, return_state=True)
    assert not S.any()
    grads = K.bwd_decay(q, q, q, q, ld, initial_state=S0, dfinal_state=2 * S0)
    assert torch.equal(grads[3], 2 * S0)
    st = S0.clone()
    K.decode_decay(q, q, q, ld, st)
    assert torch.equal(st, S0)


def test_decay_state_in_place_and_continued_prompts():
    # a prompt in three pieces, each continuing the state in place of the last one's, is the prompt
    q, k, v = (_randn(i, 2, 900, 2, 64) for i in range(3))
    ld = _decays(2)
    st, outs = None, []
    for a, b in ((0, 130), (130, 131), (131, 900)):
        o, st = K.fwd_decay(q[:, a:b], k[:, a:b], v[:, a:b], ld, initial_state=st, return_state=True)
        outs.append(o)
    _check_decay(q, k, v, ld, 1.0, o=torch.cat(outs, 1), S=st)


@pytest.mark.parametrize("T,H", [(64, 2), (700, 16), (2000, 16), (9000, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_final_state_over_the_initial_one(dtype, T, H):
    """The C entry takes one array for both states, whichever way the segments are joined."""
    q, k, v = (_randn(i, 1, T, H, 64, dtype=dtype) for i in range(3))
    cu = torch.tensor([0, T // 3, T], dtype=torch.int32, device=DEV)
    ld, st = _decays(H), _randn(5, 2, H, 64, 64)
    want_o, want = K.fwd_decay(q, k, v, ld, initial_state=st, cu_seqlens=cu, return_state=True)
    o = torch.empty_like(q)
    pr = KL._decay_problem(q, k, v, ld, 1.0, cu, o=o)
    ws = torch.empty(max(256, K.decay_workspace_size(q, k, v, ld, cu_seqlens=cu)), dtype=torch.uint8, device=DEV)
    KL._run("kata_fwd_decay", q.device, pr, q.data_ptr(), k.data_ptr(), v.data_ptr(), ld.data_ptr(), cu.data_ptr(),
            st.data_ptr(), o.data_ptr(), st.data_ptr(), ws.data_ptr(), ws.numel())
    # the scan and the walk add a state's terms in the same order and precision
    assert torch.equal(o, want_o) and torch.equal(st, want)


@pytest.mark.parametrize("lengths,H", [([100, 2000], 16), ([1, 0, 77, 2000], 16), ([2000, 64], 16),
                                       ([1, 0, 77, 512, 130, 1303], 16), ([9000, 30, 0, 1], 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decay_one_array_for_both_states_of_short_and_long_sequences(dtype, lengths, H):
    """Sequences of one segment in a call whose longer ones are joined by the scan: it writes their final
    states before the walk needs the initial ones."""
    T, n = sum(lengths), len(lengths)
    q, k, v = (_randn(i, 1, T, H, 64, dtype=dtype) for i in range(3))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)
    ld, S0 = _decays(H), _randn(5, n, H, 64, 64)
    want_o, want = K.fwd_decay(q, k, v, ld, initial_state=S0, cu_seqlens=cu, return_state=True)
    st, o = S0.clone(), torch.empty_like(q)
    pr = KL._decay_problem(q, k, v, ld, 1.0, cu, o=o)
    ws = torch.empty(K.decay_workspace_size(q, k, v, ld, cu_seqlens=cu), dtype=torch.uint8, device=DEV)
    assert ws.numel()                                # the long sequences have segments
    KL._run("kata_fwd_decay", q.device, pr, q.data_ptr(), k.data_ptr(), v.data_ptr(), ld.data_ptr(), cu.data_ptr(),
            st.data_ptr(), o.data_ptr(), st.data_ptr(), ws.data_ptr(), ws.numel())
    assert torch.equal(st, want) and torch.equal(o, want_o)
    heads = [0, H - 1]                               # the strongest and the weakest decay
    part = [x[:, :, heads] for x in (q, k, v)]
    _check_decay(*part, ld[heads], 1.0, lengths, S0=S0[:, heads], o=o[:, :, heads], S=st[:, heads])


def test_decay_large_offsets():
    # rows beyond 2^31 elements: head-major views of one big buffer, the last rows of each head used
    T, H, d = 9_000_000, 4, 64                       # 2.3e9 bf16 elements
    big = torch.empty(1, H, T, d, dtype=BF, device=DEV)
    tail = slice(T - 200, T)
    big[:, :, tail] = _randn(1, 1, H, 200, d, dtype=BF)
    x = big.transpose(1, 2)[:, tail]
    ld = _decays(H)
    assert torch.equal(K.fwd_decay(x, x, x, ld), K.fwd_decay(*[x.contiguous()] * 3, ld))


@pytest.mark.parametrize("T,dk,dv", [(2200, 64, 64), (2600, 64, 64), (2600, 128, 40), (2600, 40, 128)])
def test_decay_segments_joined_by_the_walk_and_by_the_scan(T, dk, dv):
    # 12 and 14 segments of three chunks, with all states
    q, k, v, g = (_randn(i, 1, T, 1, d, dtype=BF) for i, d in ((1, dk), (2, dk), (3, dv), (4, dv)))
    S0, dS, ld = _randn(5, 1, 1, dk, dv), _randn(6, 1, 1, dk, dv), _decays(1, "-0.004")
    o, S = K.fwd_decay(q, k, v, ld, scale=0.125, initial_state=S0, return_state=True)
    grads = K.bwd_decay(q, k, v, g, ld, scale=0.125, initial_state=S0, dfinal_state=dS)
    _check_decay(q, k, v, ld, 0.125, S0=S0, dO=g, dS=dS, o=o, S=S, grads=grads)


@pytest.mark.parametrize("dtype,B,H", [(BF, 64, 32), (F32, 64, 16)])
def test_decay_of_operands_larger_than_the_caches(dtype, B, H):
    # loaded past the caches; half of the sequences are not, and get the same results
    q, k, v = (_randn(i, B, 500, H, 64, dtype=dtype) for i in range(3))
    ld = _decays(H)
    o = K.fwd_decay(q, k, v, ld)
    for part in (slice(0, B // 2), slice(B // 2, B)):
        assert torch.equal(o[part], K.fwd_decay(q[part], k[part], v[part], ld))


def test_decay_of_more_workgroups_than_a_grid_axis_has():
    # 65535 one-token sequences of 260 heads: 17 million workgroups of 256 threads, over 2^32 work-items,
    # which one grid axis cuts off.  The sequences share their inputs, so every output row is the first one's.
    n, H, d = 65535, 260, 8
    q, k, v = (_randn(i, 1, 1, H, d, dtype=BF).expand(n, 1, H, d) for i in range(3))
    ld = _decays(H)
    o = K.fwd_decay(q, k, v, ld, scale=0.5)
    one = K.fwd_decay(q[:1], k[:1], v[:1], ld, scale=0.5)
    assert torch.equal(o, one.expand(n, 1, H, d))
    _check_decay(q[:1], k[:1], v[:1], ld, 0.5, o=one)


def test_decay_refusals():
    q, k, v = (_randn(i, 1, 8, 2, 64, dtype=BF) for i in range(3))
    ld = _decays(2)
    cu = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        K.fwd_decay(q.half(), k.half(), v.half(), ld)
    for bad in (lambda: K.fwd_decay(q, k[..., :32], v, ld), lambda: K.fwd_decay(q, k, v.float(), ld),
                lambda: K.fwd_decay(q, k, v, ld[:1]), lambda: K.fwd_decay(q, k, v, ld.double()),
                lambda: K.fwd_decay(q, k, v, ld.cpu()), lambda: K.fwd_decay(q, k, v, ld, cu_seqlens=cu.long()),
                lambda: K.fwd_decay(q, k, v, ld, cu_seqlens=cu[:1]),
                lambda: K.fwd_decay(*[x.expand(2, 8, 2, 64) for x in (q, k, v)], ld, cu_seqlens=cu),
                lambda: K.fwd_decay(q, k, v, ld, initial_state=torch.zeros(1, 2, 64, 32, device=DEV)),
                lambda: K.fwd_decay(q, k, v, ld, out=torch.empty_like(v, dtype=F32)),
                lambda: K.fwd_decay(q[..., ::2], k[..., ::2], v, ld),
                lambda: K.bwd_decay(q, k, v, v.float(), ld), lambda: K.bwd_decay(q, k, v, v[:, :4], ld),
                lambda: K.decode_decay(q, k, v, ld, torch.zeros(1, 2, 64, 64, device=DEV, dtype=BF)),
                lambda: K.decode_decay(q, k, v, ld, None),
                lambda: K.fwd_decay(*[_randn(1, 1, 999, 1, 64)] * 3, ld[:1], workspace=torch.empty(
                    1, dtype=torch.uint8, device=DEV).expand(1 << 30)),
                lambda: K.parallel_decay_attn(q, k, v, ld.clone().requires_grad_()),
                lambda: K.parallel_decay_attn(q, k, v, ld, cu_seqlens=cu, rotary=K.rotary_rates(64)),
                lambda: K.parallel_decay_attn(q, k, v, ld, norm=(torch.ones(32, device=DEV), None))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: K.fwd_decay(*[x[..., :12].contiguous() for x in (q, k, v)], ld),   # 24-byte rows
                lambda: K.fwd_decay(*[torch.zeros(1, 8, 2, 136, device=DEV, dtype=BF)] * 3, ld),
                lambda: K.fwd_decay(q, k, v, ld, scale=float("nan")),
                lambda: K.fwd_decay(q.view(-1)[4:964].view(1, 15, 1, 64), *[q.view(-1)[:960].view(1, 15, 1, 64)] * 2, ld[:1]),
                lambda: K.fwd_decay(*[_randn(1, 1, 999, 1, 64)] * 3, ld[:1],
                                    workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(K.KataError):
            bad()


# ---- rotary positions --------------------------------------------------------------------------

@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,H,Hk,D,rot", [(1, 1, 1, 1, 2, 2), (2, 3, 2, 1, 64, 64), (3, 17, 4, 2, 80, 48),
                                            (1, 130, 3, 3, 33, 6), (2, 5, 2, 1, 128, 0), (1, 9, 1, 1, 24, 24),
                                            (4, 1, 16, 16, 64, 64), (1, 3, 2, 2, 40, 18), (1, 2, 1, 1, 1024, 1024)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary(dtype, B, T, H, Hk, D, rot, interleaved, inverse):
    q, k = _randn(1, B, T, H, D, dtype=dtype), _randn(2, B, T, Hk, D, dtype=dtype)
    rates = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).to(DEV)
    start = torch.arange(B)[:, None] * 250000 + 3
    pos = (start + torch.arange(T)).to(DEV)
    kw = dict(interleaved=interleaved, magnitude=1.25, inverse=inverse)
    got = K.rotary(q, k, rates, positions=pos, **kw)
    for x, y in zip((q, k), got):
        ref = L.rotary(_np(x), _np(pos), _np(rates), interleaved, 1.25, inverse)
        size = np.zeros_like(ref)                    # |a| + |b| of the turned pairs
        n = rot // 2
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, n), slice(n, rot))
        size[..., a] = size[..., b] = np.abs(_np(x)[..., a]) + np.abs(_np(x)[..., b])
        turned = np.zeros(D, dtype=bool)
        turned[:rot] = True
        tol = 1.25 * 2.0 ** -21 * size + np.where(turned, U[dtype] * 1.01, 0.0) * np.abs(ref)
        _inside(y, ref, tol, "rotary")               # what is copied is the same to the bit
    # other ways to say the same: in place, int32 positions, one tensor, broadcast positions
    a, b = q.clone(), k.clone()
    K.rotary(a, b, rates, positions=pos.int(), out=(a, b), **kw)
    assert torch.equal(a, got[0]) and torch.equal(b, got[1])
    assert torch.equal(K.rotary(q, None, rates, positions=pos, **kw), got[0])
    row = K.rotary(q, k, rates, positions=pos[:1], **kw)
    assert torch.equal(row[0][0], got[0][0])
    off = K.rotary(q, k, rates, offset=3, **kw)
    assert torch.equal(off[0], row[0])


@pytest.mark.parametrize("H,Hk", [(2, 0), (0, 2), (0, 0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_without_heads_on_one_side(dtype, H, Hk):
    q, k = _randn(1, 2, 5, H, 16, dtype=dtype), _randn(2, 2, 5, Hk, 16, dtype=dtype)
    rates, m = K.rotary_rates(16)
    want = [K.rotary(x, None, rates, offset=7) if x.numel() else x for x in (q, k)]
    outs = torch.zeros_like(q), torch.zeros_like(k)
    got = K.rotary(q, k, rates, offset=7, out=outs)
    assert got[0] is outs[0] and got[1] is outs[1]
    for got in (got, K.rotary(q, k, rates, offset=7)):
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    leaves = q.clone().requires_grad_(), k.clone().requires_grad_()
    a, b = KL.turn(*leaves, (rates, m), offset=7)
    grads = torch.autograd.grad(a.sum() + b.sum(), leaves)
    for x, g in zip((q, k), grads):
        ones = torch.ones_like(x)
        assert torch.equal(g, K.rotary(ones, None, rates, offset=7, inverse=True) if x.numel() else x)


def test_rotary_strides_and_alignment():
    fused = _randn(1, 2, 7, 3, 200, dtype=BF)
    rates, m = K.rotary_rates(64)
    for lo in (0, 8, 1, 3):                          # rows aligned to 16 bytes, and not
        x = fused[..., lo:lo + 64]
        out = torch.zeros_like(fused)
        y = K.rotary(x, None, rates, out=out[..., lo:lo + 64])
        assert torch.equal(y, K.rotary(x.contiguous(), None, rates))
        assert not out[..., :lo].any() and not out[..., lo + 64:].any()
    x = fused[..., :64]
    assert torch.equal(K.rotary(x[:1].expand(2, 7, 3, 64), None, rates)[1], K.rotary(x, None, rates)[0])
    assert torch.equal(K.rotary(x.transpose(1, 2).contiguous().transpose(1, 2), None, rates), K.rotary(x, None, rates))


def test_rotary_negative_and_far_positions():
    x = _randn(1, 1, 4, 1, 16)
    pos = torch.tensor([[-5, 0, 2 ** 31 + 11, 10 ** 9]], device=DEV)
    rates, _ = K.rotary_rates(16)
    ref = L.rotary(_np(x), _np(pos), _np(rates))
    # an angle of 2^31 is known to 2^31 2^-52 in fp64, on both sides
    _inside(K.rotary(x, None, rates, positions=pos), ref, 2.0 ** -19 * np.abs(_np(x)).sum(-1, keepdims=True), "far")


def test_rotary_of_more_workgroups_than_a_grid_axis_has():
    # a workgroup a token, 16.8 million of them; every token is the same one at another position
    T, H = (1 << 24) + 20000, 257
    q = _randn(1, 1, 1, H, 2, dtype=BF).expand(1, T, H, 2)
    rates, m = K.rotary_rates(2, base=100.0)
    out = torch.full((1, T, H, 2), float("nan"), dtype=BF, device=DEV)
    K.rotary(q, None, rates * 1e-3, out=out)
    for at in range(0, T, 1 << 21):
        assert not torch.isnan(out[:, at:at + (1 << 21)]).any(), at
    for at in (0, 19000, 1 << 22, (1 << 23) - 7, (1 << 24) - 500, T - 1000):
        assert torch.equal(out[:, at:at + 1000], K.rotary(q[:, :1000], None, rates * 1e-3, offset=at)[:, :T - at]), at


def test_rotary_refusals():
    q, k = _randn(1, 1, 4, 2, 16), _randn(2, 1, 4, 1, 16)
    rates, _ = K.rotary_rates(16)
    for bad in (lambda: K.rotary(q, k[:, :2], rates), lambda: K.rotary(q, k.bfloat16(), rates),
                lambda: K.rotary(q, k, rates.float()), lambda: K.rotary(q, k, rates.cpu()),
                lambda: K.rotary(q[..., :8], k[..., :8], rates), lambda: K.rotary(q, k, rates, positions=q[0, :, 0, 0]),
                lambda: K.rotary(q, k, rates, positions=torch.zeros(3, dtype=torch.int64, device=DEV)),
                lambda: K.rotary(q, k, rates, out=q), lambda: K.rotary(q[..., ::2], None, rates[:4])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        K.rotary(q.double(), None, rates)
    with pytest.raises(K.KataError):
        K.rotary(torch.zeros(1, 1, 1, 2000, device=DEV), None, rates)


# ---- layer norm ---------------------------------------------------------------------------------

WIDTHS = [1, 2, 7, 8, 24, 64, 65, 100, 128, 200, 256, 500, 512, 513, 1000, 1024, 1536, 2048, 2049, 4096, 6000,
          8192, 8200, 10000, 16392]


def _norm_chain(N):
    return N + 8 if N < 64 else 72 + N / 256


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype,wtype", [(BF, F32), (BF, BF), (F32, F32), (BF, None)])
def test_layer_norm(dtype, wtype, N):
    rows = 37 if N <= 2048 else 5
    print("case", dtype, wtype, N, flush=True)
    x, dy = _randn(1, rows, N, dtype=dtype) + 0.5, _randn(2, rows, N, dtype=dtype)
    w, b = (None, None) if wtype is None else (_randn(3, N, dtype=wtype), _randn(4, N, dtype=wtype))
    y, mean, rstd = K.fwd_layer_norm(x, w, b, eps=1e-3, return_stats=True)
    nx, ndy = _np(x), _np(dy)
    nw, nb = (None, None) if w is None else (_np(w), _np(b))
    ry, rm, rr = L.layer_norm(nx, nw, nb, 1e-3)
    c = _norm_chain(N) * 2.0 ** -24
    em = (c * np.abs(nx).mean(-1) + 2.0 ** -24 * np.abs(rm))
    _inside(mean, rm, em, "mean")
    # the variance of differences that are off by em: relative c + 2 em / sd, half of it in rstd
    er = rr * (c + 2.0 ** -22 + em * rr)
    _inside(rstd, rr, er, "rstd")
    hat = (nx - rm[:, None]) * rr[:, None]
    eh = rr[:, None] * (em[:, None] + 2.0 ** -24 * np.abs(nx)) + np.abs(hat) * (er / rr + 2.0 ** -22)[:, None]
    aw = 1.0 if nw is None else np.abs(nw)
    _inside(y, ry, aw * eh + (U[dtype] * 1.01 + 2.0 ** -23) * np.abs(ry) + 2.0 ** -22 * aw * np.abs(hat), "y")
    assert torch.equal(K.fwd_layer_norm(x, w, b, eps=1e-3), y)

    dx, dw, db = K.bwd_layer_norm(dy, x, w, mean, rstd)
    rdx, rdw, rdb = L.layer_norm_backward(ndy, nx, nw, 1e-3)
    t = ndy if nw is None else ndy * nw
    at, ah = np.abs(t), np.abs(hat)
    m1, m2 = at.mean(-1, keepdims=True), (at * ah).mean(-1, keepdims=True)
    # every term of dx with its relative error, and the error of hat in the two places it enters
    e = (4 * c + 2.0 ** -21) * (at + m1 + ah * m2) + eh * m2 + ah * (at * eh).mean(-1, keepdims=True)
    tol = rr[:, None] * e + (er / rr)[:, None] * np.abs(rdx) + (U[dtype] * 1.01) * np.abs(rdx)
    _inside(dx, rdx, tol, "dx")
    uw = U[BF] * 1.01 if wtype == BF else 2.0 ** -24
    _inside(dw, rdw, (np.abs(ndy) * (eh + (rows + 64) * 2.0 ** -24 * ah)).sum(0) + uw * np.abs(rdw), "dw")
    _inside(db, rdb, (rows + 64) * 2.0 ** -24 * np.abs(ndy).sum(0) + uw * np.abs(rdb), "db")
    again = K.bwd_layer_norm(dy, x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    assert K.bwd_layer_norm(dy, x, w, mean, rstd, params=False)[1:] == (None, None)


@pytest.mark.parametrize("N", [64, 1000, 1024])
def test_layer_norm_many_rows(N):
    # more rows than the workgroups of a launch take at once; sums over all of them
    rows = 40000 if N == 64 else 9001
    x, dy = _randn(1, rows, N, dtype=BF), _randn(2, rows, N, dtype=BF)
    w = _randn(3, N)
    y, mean, rstd = K.fwd_layer_norm(x, w, None, return_stats=True)
    dx, dw, db = K.bwd_layer_norm(dy, x, w, mean, rstd)
    nx, ndy, nw = _np(x), _np(dy), _np(w)
    ry, rm, rr = L.layer_norm(nx, nw)
    rdx, rdw, rdb = L.layer_norm_backward(ndy, nx, nw)
    hat = np.abs((nx - rm[:, None]) * rr[:, None])
    # fp32 arithmetic is off by far less than a bf16 step of the largest term here
    _inside(y, ry, U[BF] * 1.01 * np.abs(ry) + 2.0 ** -16 * (hat + 1) * np.abs(nw), "y")
    t = np.abs(ndy * nw)
    _inside(dx, rdx, U[BF] * 1.01 * np.abs(rdx) + 2.0 ** -16 * rr[:, None] * (t + t.mean(-1, keepdims=True) * (1 + hat)), "dx")
    # a sum runs over its workgroup's rows (at most rows / 1024 + 1 a lane group), 1024 partial ones in
    # 16 slices, and the tree: under 256 additions
    _inside(dw, rdw, (256 * 2.0 ** -24 + 2.0 ** -17) * (np.abs(ndy) * (hat + 1)).sum(0), "dw")
    _inside(db, rdb, 256 * 2.0 ** -24 * np.abs(ndy).sum(0), "db")


@pytest.mark.parametrize("N", [8192, 8193, 8200])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layer_norm_gradients_stay_inside_their_workspace(dtype, N):
    # more rows than workgroups keep sums of; the bytes behind the workspace are left alone
    rows = 900
    x, dy = _randn(1, rows, N, dtype=dtype), _randn(2, rows, N, dtype=dtype)
    _, mean, rstd = K.fwd_layer_norm(x, return_stats=True)
    need = K.layer_norm_workspace_size(x)
    ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device=DEV)
    dx, dw, db = K.bwd_layer_norm(dy, x, None, mean, rstd, workspace=ws[:need])
    assert (ws[need:] == 171).all()
    hat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    _inside(dw, _np((dy.double() * hat).sum(0)), _np((rows + 64) * 2.0 ** -23 * (dy.double() * hat).abs().sum(0)), "dw")
    _inside(db, _np(dy.double().sum(0)), _np((rows + 64) * 2.0 ** -24 * dy.double().abs().sum(0)), "db")


def test_layer_norm_strides_in_place_and_empty():
    big = _randn(1, 6, 5, 200, dtype=BF)
    for lo in (0, 8, 3):
        x = big[..., lo:lo + 128]
        want = K.fwd_layer_norm(x.contiguous())
        assert torch.equal(K.fwd_layer_norm(x), want)
        a = big.clone()
        K.fwd_layer_norm(a[..., lo:lo + 128], out=a[..., lo:lo + 128])
        assert torch.equal(a[..., lo:lo + 128], want)
        assert torch.equal(a[..., :lo], big[..., :lo]) and torch.equal(a[..., lo + 128:], big[..., lo + 128:])
    t = big.transpose(0, 1)
    assert torch.equal(K.fwd_layer_norm(t), K.fwd_layer_norm(t.contiguous()))
    e = torch.empty(0, 4, 64, device=DEV)
    y, mean, rstd = K.fwd_layer_norm(e, return_stats=True)
    dx, dw, db = K.bwd_layer_norm(e, e, None, mean, rstd)
    assert y.shape == e.shape and dx.shape == e.shape and not dw.any() and not db.any()
    const = torch.full((3, 96), 2.5, device=DEV)
    assert not K.fwd_layer_norm(const).any()         # no variance: zero
    bad = _randn(2, 4, 64)
    bad[1, 3] = float("nan")
    bad[2, 0] = float("inf")
    y = K.fwd_layer_norm(bad)
    assert torch.isfinite(y[[0, 3]]).all() and not torch.isfinite(y[1]).any()


def test_layer_norm_forward_needs_no_strides_of_gradients():
    x, y = _randn(1, 5, 64), torch.empty(5, 64, device=DEV)
    pr = KL._NORM.pack(5, 64, KL._dtype(F32), KL._dtype(F32), 1e-5, 64, 0, 64, 0)
    KL._run("kata_fwd_layer_norm", x.device, pr, x.data_ptr(), None, None, y.data_ptr(), None, None)
    assert torch.equal(y, K.fwd_layer_norm(x))


@pytest.mark.parametrize("step", [1, 3, 64])
def test_layer_norm_of_windows_that_overlap(step):
    base = _randn(1, 2, 200)
    x = base.unfold(1, 64, step)                     # (2, windows, 64), rows `step` elements apart
    dy = _randn(2, 2, 200).unfold(1, 64, step)
    y, mean, rstd = K.fwd_layer_norm(x, return_stats=True)
    assert torch.equal(y, K.fwd_layer_norm(x.contiguous()))
    got, want = K.bwd_layer_norm(dy, x, None, mean, rstd), K.bwd_layer_norm(dy.contiguous(), x.contiguous(), None, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(K.fwd_layer_norm(x[0]), y[0]) and torch.equal(K.fwd_layer_norm(x[0, :1]), y[0, :1])


def test_layer_norm_refusals():
    x, w = _randn(1, 4, 64, dtype=BF), torch.ones(64, device=DEV)
    mean = torch.zeros(4, device=DEV)
    for bad in (lambda: K.fwd_layer_norm(x, w[:32]), lambda: K.fwd_layer_norm(x, w, w.bfloat16()),
                lambda: K.fwd_layer_norm(x, w.cpu()), lambda: K.fwd_layer_norm(x, out=x[:2]),
                lambda: K.fwd_layer_norm(x[:, :0]), lambda: K.bwd_layer_norm(x.float(), x, w, mean, mean),
                lambda: K.bwd_layer_norm(x, x, w, mean[:2], mean), lambda: K.bwd_layer_norm(x, x, w, mean, mean.double()),
                lambda: K.fwd_layer_norm(x, out=torch.empty(64, 4, device=DEV, dtype=BF).t())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        K.fwd_layer_norm(x.half())
    with pytest.raises(K.KataError):
        K.fwd_layer_norm(x.float(), w.bfloat16())
    with pytest.raises(K.KataError):
        K.fwd_layer_norm(x, w, eps=-1.0)


# ---- the operators together ------------------------------------------------------------------------

def test_one_layer_prompt_then_tokens():
    # rotary -> decayed attention -> norm over all heads: a prompt, then single tokens, against one pass
    # of the oracle over the whole sequence
    B, T, n, H, d = 2, 150, 4, 2, 64
    q, k, v = (_randn(i, B, T + n, H, d) for i in range(3))
    ld, (rates, m) = _decays(H), K.rotary_rates(d, scaling="parts", factor=4.0, original_length=64)
    w, b = _randn(5, H * d), _randn(6, H * d)
    y, st = K.parallel_decay_attn(q[:, :T], k[:, :T], v[:, :T], ld, scale=0.125, return_state=True, rotary=(rates, m), norm=(w, b))
    ys = [y]
    for t in range(T, T + n):
        qt, kt = K.rotary(q[:, t:t + 1], k[:, t:t + 1], rates, offset=t, magnitude=m)
        o = K.decode_decay(qt, kt, v[:, t:t + 1], ld, st, scale=0.125)
        ys.append(K.layer_norm(o.flatten(2), w, b).view(o.shape))
    got = torch.cat(ys, 1)
    pos = np.broadcast_to(np.arange(T + n), (B, T + n))
    rq, rk = (L.rotary(_np(x), pos, _np(rates), magnitude=m) for x in (q, k))
    size_q, size_k = (np.abs(_np(x)).max() * 2 * m for x in (q, k))
    o, size = np.zeros((B, T + n, H, d)), np.zeros((B, T + n, H, d))
    for i in range(B):
        for h in range(H):
            a = [x[i, :, h] for x in (rq, rk, _np(v))]
            o[i, :, h] = L.decay_closed(*a, _np(ld)[h], 0.125)[0]
            size[i, :, h] = L.decay_closed(*[np.abs(x) for x in a], _np(ld)[h], 0.125)[0]
            # the turned q and k are off by 2^-21 of their largest pair: a row of 64 of them
            W = L.decay_weights(_np(ld)[h], T + n)
            size[i, :, h] += 0.125 * 2 * d * size_q * size_k * (W @ np.abs(_np(v)[i, :, h]))
    e = ((2 * T + d + 64) * 2.0 ** -24 + 8 * 2.0 ** -21) * size.reshape(B, T + n, -1)
    ry, rm, rr = L.layer_norm(o.reshape(B, T + n, -1), _np(w), _np(b))
    hat = np.abs((o.reshape(B, T + n, -1) - rm[..., None]) * rr[..., None])
    moved = rr[..., None] * (e + e.mean(-1, keepdims=True) + hat * np.sqrt((e * e).mean(-1, keepdims=True)) * 1.01)
    _inside(got.flatten(2), ry, np.abs(_np(w)) * (moved + 80 * 2.0 ** -24 * (hat + 1)) + 2.0 ** -22 * np.abs(ry), "layer")


@pytest.mark.parametrize("packed", [False, True])
def test_autograd_of_a_layer(packed):
    # gradients of the whole run against torch float64 autograd of the recurrence
    B, T, H, d = (1, 90, 2, 32) if packed else (2, 45, 2, 32)
    lengths = [40, 0, 50] if packed else [45, 45]
    ld, (rates, m) = _decays(H), K.rotary_rates(16)
    w, b = _randn(5, d), _randn(6, d)
    q, k, v, g = (_randn(i, B, T, H, d) for i in range(4))
    S0, gS = _randn(7, len(lengths), H, d, d), _randn(8, len(lengths), H, d, d)
    pos = torch.cat([torch.arange(n) for n in lengths]).view(B, T).to(DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV) if packed else None
    leaves = [x.clone().requires_grad_() for x in (q, k, v, S0, w, b)]
    y, st = K.parallel_decay_attn(*leaves[:3], ld, scale=0.5, initial_state=leaves[3], return_state=True,
                                  cu_seqlens=cu, rotary=(rates, m), positions=pos, interleaved=True,
                                  norm=(leaves[4], leaves[5]))
    got = torch.autograd.grad((y * g).sum() + (st * gS).sum(), leaves)

    ref = [x.detach().double().cpu().requires_grad_() for x in leaves]
    angle = pos.cpu().double()[..., None, None] * rates.cpu()

    def turned(x):
        a, c = x[..., 0:16:2], x[..., 1:16:2]
        z = torch.stack([a * angle.cos() - c * angle.sin(), a * angle.sin() + c * angle.cos()], -1).flatten(-2)
        return torch.cat([z, x[..., 16:]], -1).reshape(-1, H, d)

    tq, tk, tv = turned(ref[0]), turned(ref[1]), ref[2].reshape(-1, H, d)
    gam, at, loss = torch.exp(ld.cpu().double())[:, None, None], 0, 0.0
    for i, n in enumerate(lengths):
        S = ref[3][i]
        for t in range(at, at + n):
            S = gam * S + tk[t][:, :, None] * tv[t][:, None, :]
            o = 0.5 * (tq[t][:, :, None] * S).sum(1)
            o = torch.nn.functional.layer_norm(o, (d,), ref[4], ref[5])
            loss = loss + (o * g.cpu().double().reshape(-1, H, d)[t]).sum()
        at += n
        loss = loss + (S * gS[i].cpu().double()).sum()
    want = torch.autograd.grad(loss, ref)
    for name, x, r in zip("q k v S0 w b".split(), got, want):
        # a chain of fp32 operators: 2^-24 times the depth of their sums (under 512 additions), relative to
        # the gradient's largest entry, which the norm's backward spreads over a row
        _inside(x, r.numpy(), 512 * 2.0 ** -24 * float(r.abs().max()), name)


@pytest.mark.parametrize("B,T,H", [(0, 5, 2), (2, 0, 2), (0, 0, 2), (2, 5, 0)])
@pytest.mark.parametrize("over", ["head", "token", "none", "no norm"])
def test_a_layer_of_an_empty_batch(B, T, H, over):
    d = 32
    leaves = [torch.empty(B, T, H, d, device=DEV, requires_grad=True) for _ in range(3)]
    n = H * d if over == "token" else d
    w, b = (torch.ones(n, device=DEV, requires_grad=True) for _ in range(2))
    norm = {"none": (None, None), "no norm": None}.get(over, (w, b))
    run = lambda: K.parallel_decay_attn(*leaves, torch.zeros(H, device=DEV), rotary=K.rotary_rates(d), norm=norm)  # noqa: E731
    if n == 0:                                       # a norm over nothing
        with pytest.raises(ValueError):
            run()
        return
    o = run()
    assert o.shape == (B, T, H, d)
    grads = torch.autograd.grad(o.sum(), leaves + ([w, b] if over in ("head", "token") else []))
    assert all(g.shape == x.shape for g, x in zip(grads, leaves)) and not any(g.any() for g in grads[3:])


def test_shared_heads_and_unused_outputs_under_autograd():
    B, T, H, d = 1, 70, 4, 64
    q, k, v, ld = _randn(1, B, T, H, d), _randn(2, B, T, 1, d), _randn(3, B, T, 1, d), _decays(H)
    kl, vl = k.clone().requires_grad_(), v.clone().requires_grad_()
    o, st = K.parallel_decay_attn(q, kl.expand(B, T, H, d), vl.expand(B, T, H, d), ld, return_state=True)
    dk, dv = torch.autograd.grad(o.sum(), (kl, vl), retain_graph=True)      # dO is a broadcast one
    _, fk, fv, _ = K.bwd_decay(q, k.expand(B, T, H, d), v.expand(B, T, H, d), torch.ones_like(q), ld)
    assert torch.equal(dk, fk.sum(2, keepdim=True)) and torch.equal(dv, fv.sum(2, keepdim=True))
    sk, = torch.autograd.grad(st.sum(), kl)                                  # only the state is used
    ref = np.zeros((T, d))
    for h in range(H):
        left = np.exp(_np(ld)[h] * (T - 1 - np.arange(T)))[:, None]
        ref += left * _np(v)[0, :, 0].sum(-1, keepdims=True)
    _inside(sk[0, :, 0], ref, 2.0 ** -16 * np.abs(_np(v)).sum(), "dk of the state")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_that_arrive_at_any_alignment(dtype):
    # the gradient of a concatenation is a view at the place that its input had: contiguous, but not
    # on a 16-byte boundary
    q, k, v = (_randn(i, 1, 70, 2, 64, dtype=dtype) for i in range(3))
    ld, S0 = _decays(2), _randn(4, 1, 2, 64, 64)
    lead, c, cs = torch.zeros(1, dtype=dtype, device=DEV), _randn(5, 1 + v.numel(), dtype=dtype), _randn(6, 1 + S0.numel())
    leaves = [x.clone().requires_grad_() for x in (q, k, v, S0)]
    o, S = K.parallel_decay_attn(*leaves[:3], ld, initial_state=leaves[3], return_state=True)
    loss = (torch.cat([lead, o.flatten()]) * c).sum() + (torch.cat([lead.float(), S.flatten()]) * cs).sum()
    got = torch.autograd.grad(loss, leaves)
    want = K.bwd_decay(q, k, v, c[1:].clone().view_as(v), ld, initial_state=S0, dfinal_state=cs[1:].clone().view_as(S0))
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_kata_attention_with_rotary():
    q, k, v = (_randn(i, 1, 128, 2, d, dtype=BF) for i, d in ((1, 16), (2, 16), (3, 64)))
    table = K.rotary_rates(16)
    a, b = K.rotary(q, k, table[0])
    assert torch.equal(K.parallel_kata_attn(q, k, v, rotary=table), K.parallel_kata_attn(a, b, v))


def test_tensors_written_in_place_tell_autograd():
    q, k, v = (_randn(i, 2, 3, 2, 64) for i in range(3))
    ld, (rates, _) = _decays(2), K.rotary_rates(64)
    st = _randn(4, 2, 2, 64, 64)
    o, a, b, y = (torch.empty_like(q) for _ in range(4))
    for call, written in ((lambda: K.decode_decay(q, k, v, ld, st), [st]),
                          (lambda: K.decode_decay(q, k, v, ld, st, out=o), [st, o]),
                          (lambda: K.fwd_decay(q, k, v, ld, out=o), [o]),
                          (lambda: K.rotary(q, k, rates, out=(a, b)), [a, b]),
                          (lambda: K.rotary(q, None, rates, out=a), [a]),
                          (lambda: K.fwd_layer_norm(q, out=y), [y])):
        reads = q._version, k._version, v._version, ld._version
        before = [x._version for x in written]
        call()
        assert all(x._version > n for x, n in zip(written, before))
        assert reads == (q._version, k._version, v._version, ld._version)
    # a state that a backward pass still needs, advanced by a token
    leaf = q.clone().requires_grad_()
    loss = K.parallel_decay_attn(leaf, k, v, ld, initial_state=st).sum()
    K.decode_decay(q, k, v, ld, st)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    with torch.inference_mode():                     # whose tensors have no counters
        s = st.clone()
        K.decode_decay(q, k, v, ld, s, out=torch.empty_like(v))
        K.rotary(q, k, rates, out=(torch.empty_like(q), torch.empty_like(k)))
        K.fwd_layer_norm(q, out=torch.empty_like(q))
    K.decode_decay(q, k, v, ld, st)
    assert torch.equal(s, st)


def test_timing_records_every_kernel_of_a_layer():
    q, k, v, g = (_randn(i, 1, 900, 2, 64, dtype=BF) for i in range(4))
    ld, (rates, _) = _decays(2), K.rotary_rates(64)
    w = torch.ones(64, device=DEV)
    K.fwd_decay(q, k, v, ld)
    K.timing_begin()
    K.rotary(q, k, rates)
    o = K.fwd_decay(q, k, v, ld)
    y, mean, rstd = K.fwd_layer_norm(o, w, return_stats=True)
    K.bwd_layer_norm(g, o, w, mean, rstd)
    K.bwd_decay(q, k, v, g, ld)
    t = K.timing_end()
    assert set(t) == set(K.KERNEL_KINDS)
    assert t["rotary"][0] == 1 and t["norm"][0] == 2 and t["chunk_output"][0] == 1 and t["bwd"][0] == 1
    assert all(ms > 0 for n, ms in t.values() if n)
    K.rotary(q, k, rates)                            # recording has stopped
    K.timing_begin()
    assert not any(n for n, _ in K.timing_end().values())


def test_side_stream():
    s = torch.cuda.Stream()
    q, k, v = (_randn(i, 1, 1000, 2, 64, dtype=BF) for i in range(3))
    ld, (rates, m) = _decays(2), K.rotary_rates(64)
    want = K.parallel_decay_attn(q, k, v, ld, rotary=(rates, m), norm=(None, None))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = K.parallel_decay_attn(q, k, v, ld, rotary=(rates, m), norm=(None, None))
    s.synchronize()
    assert torch.equal(got, want)


def test_replays_of_captured_graphs():
    # two graphs of a training step and of a decode step, replayed in turn with eager work between
    q, k, v, g = (_randn(i, 1, 900, 2, 64, dtype=BF) for i in range(4))
    ld, (rates, m) = _decays(2), K.rotary_rates(64)
    w, b = _randn(5, 64), _randn(6, 64)
    tok = [_randn(i, 3, 1, 2, 64, dtype=BF) for i in (7, 8, 9)]
    st = _randn(10, 3, 2, 64, 64)

    def train():
        a, c = K.rotary(q, k, rates, magnitude=m)
        o, S = K.fwd_decay(a, c, v, ld, return_state=True)
        y, mean, rstd = K.fwd_layer_norm(o, w, b, return_stats=True)
        dx, dw, db = K.bwd_layer_norm(g, o, w, mean, rstd)
        return (y, S, dw, db, *K.bwd_decay(a, c, v, dx, ld)[:3])

    def step():
        a, c = K.rotary(tok[0], tok[1], rates, offset=5)
        return K.fwd_layer_norm(K.decode_decay(a, c, tok[2], ld, st), w, b)

    train(), K.decode_decay(*tok, ld, st.clone())
    torch.cuda.synchronize()
    graphs, outs = [], []
    S0 = st.clone()
    for f in (train, step):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = f()
        graphs.append(gr), outs.append(out)
    st.copy_(S0)
    ref = S0.clone()
    for i in range(4):
        for x, j in zip((q, k, v, g), range(4)):
            x.copy_(_randn(20 + 4 * i + j, 1, 900, 2, 64, dtype=BF))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs[0]], outs[1].clone(), st.clone()
        want = train()
        assert all(torch.equal(x, y) for x, y in zip(got[0], want))
        st.copy_(ref)
        y = step()
        assert torch.equal(got[1], y) and torch.equal(got[2], st)
        ref = st.clone()
