"""The gated delta rule, the norm of queries and keys with their rotation, and positions of several axes on the GPU
against the fp64 oracle.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24; u is what an operand that
comes out of fp32 sums holds (two bf16 terms: 2^-18, three: 2^-27; fp32 2^-24).
  delta rule: with keys of unit length and beta in [0, 1] a token maps the state by a contraction, so errors add up and
    do not grow.  M is the largest 2-norm that a column of the state has along the sequence, plus the largest |v|
    (delta_sizes).  A chunk rounds at most eight operands (the state, the inverse, the correction before and after
    it, the weights of the pairs, q's part of the state) of size M at most, and sums at most dk + 2 64 terms in
    fp32; a state is off by (chunks + 1) (8 u + (dk + 128) 2^-24) M, an output by |q| scale times as much and its
    own rounding.  The inverse's two terms are 2^-18 of its entries off the diagonal also where u is 2^-27.
  dq, dk: a term of their chunked forms (delta_gradient_sizes) has at most two factors rounded to bf16, the result
    one rounding; dv and dbeta come out of the recurrence in reversed time, like an output, with |K D| for a column.
    dlog_decay is a sum of terms with the absolute sum Bl, each good to 16 u, two bf16 terms of the pairs' weights.
  norms: the sum of squares runs over at most 16 additions a lane and 6 levels; sine and cosine are good to 2^-21 of
    a coordinate pair (as for rotary).
"""

import numpy as np
import pytest
import torch

import kernelized_psd_feature_amd as K
from oracle import delta_oracle as O

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


def _unit(seed, *shape, dtype=F32):
    x = _randn(seed, *shape)
    # a little short of one, so that rounding to bf16 leaves it so
    return (x * (0.99 / x.norm(dim=-1, keepdim=True))).to(dtype)


def _inside(got, ref, tol, what):
    g = _np(got) if torch.is_tensor(got) else got
    bad = ~(np.abs(g - ref) <= tol + 1e-30)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(g - ref) - tol, -1.0)), g.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {g.size} off, worst at {at}: {g[at]} for {ref[at]}, "
                             f"tolerance {np.broadcast_to(tol, g.shape)[at]}")
    print(f"{what}: worst share of the tolerance {np.max(np.abs(g - ref) / (tol + 1e-30), initial=0.0):.3f}", flush=True)


def _inputs(seed, B, T, Hk, H, dk, dv, dtype, gated=True, N=None):
    q, k = _randn(seed, B, T, Hk, dk, dtype=dtype), _unit(seed + 1, B, T, Hk, dk, dtype=dtype)
    v, b = _randn(seed + 2, B, T, H, dv, dtype=dtype), torch.sigmoid(_randn(seed + 3, B, T, H)).to(dtype)
    ld = None
    if gated:                                        # memories of a token to some hundred, by head
        window = 2.0 ** -(torch.arange(H, device=DEV, dtype=torch.float32) % 9)
        ld = -window * torch.rand(B, T, H, generator=torch.Generator().manual_seed(seed + 4)).to(DEV)
    return q, k, v, b, ld, _randn(seed + 5, N or B, H, dk, dv)


def _heads(q, k, v, b, ld, rows):
    """Per (sequence, head): numpy operands."""
    q, k, v, b = (_np(x) for x in (q, k, v, b))
    ld = np.zeros(b.shape) if ld is None else _np(ld)
    share = v.shape[2] // q.shape[2]
    for i, (bb, at, n) in enumerate(rows):
        for h in range(v.shape[2]):
            s = slice(at, at + n)
            yield i, h, bb, s, (q[bb, s, h // share], k[bb, s, h // share], v[bb, s, h], b[bb, s, h], ld[bb, s, h])


def _rows(B, T, lengths=None):
    if lengths is None:
        return [(i, 0, T) for i in range(B)]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    return [(0, int(cu[i]), int(n)) for i, n in enumerate(lengths)]


def _cu(lengths, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]) + first, dtype=torch.int32, device=DEV)


def _step(n, dk, dtype, fine=False):
    """Error of a state after n tokens, in units of M."""
    u = 2.0 ** -18 if dtype == BF else 2.0 ** -24
    # fine: three terms of everything but the inverse
    per = (2 * u + 6 * 2.0 ** -27 if fine and dtype == BF else 8 * u) + (dk + 128) * 2.0 ** -24
    return ((n + 63) // 64 + 1) * per


def _check_forward(args, rows, scale, S0, o, S, dtype, oracle=O.delta_recurrent):
    dk = args[0].shape[-1]
    for i, h, b, s, (q, k, v, be, ld) in _heads(*args, rows):
        first = None if S0 is None else _np(S0)[i, h]
        ref, refS = oracle(q, k, v, be, ld, scale, first)
        M = O.delta_sizes(q, k, v, be, ld, first)
        n = len(q)
        if o is not None and n:
            tol = U[dtype] * 1.01 * np.abs(ref) + abs(scale) * np.linalg.norm(q, axis=1, keepdims=True) * M * _step(n, dk, dtype)
            _inside(o[b, s, h], ref, tol, f"o {i} {h}")
        if S is not None:
            _inside(S[i, h], refS, M * _step(n, dk, dtype, fine=True) + 2.0 ** -24 * np.abs(refS), f"state {i} {h}")


SHAPES = [(1, 1, 1, 1, 64, 64), (2, 2, 1, 2, 64, 64), (1, 63, 1, 1, 32, 32), (1, 64, 2, 2, 64, 64), (2, 65, 1, 3, 64, 64),
          (1, 130, 1, 1, 16, 8), (1, 200, 2, 2, 128, 128), (1, 200, 1, 2, 64, 128), (1, 200, 1, 1, 128, 40), (1, 300, 3, 3, 24, 72),
          (2, 700, 1, 1, 40, 104), (1, 1000, 2, 2, 64, 64), (1, 1000, 1, 1, 128, 128)]


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_forward(dtype, shape, states):
    B, T, Hk, H, dk, dv = shape
    *args, S0 = _inputs(sum(shape), *shape, dtype)
    if states:
        o, S = K.fwd_delta(*args, scale=0.25, initial_state=S0, return_state=True)
    else:
        o, S, S0 = K.fwd_delta(*args, scale=0.25), None, None
    _check_forward(args, _rows(B, T), 0.25, S0, o, S, dtype)


@pytest.mark.parametrize("T,dk,dv", [(1, 4, 4), (70, 12, 20), (300, 100, 68), (130, 36, 124), (200, 4, 128), (130, 128, 4)])
def test_delta_fp32_widths_of_odd_vectors(T, dk, dv):
    *args, S0 = _inputs(T + dk, 1, T, 1, 2, dk, dv, F32)
    o, S = K.fwd_delta(*args, initial_state=S0, return_state=True)
    _check_forward(args, _rows(1, T), 1.0, S0, o, S, F32)
    _check_backward(args, _rows(1, T), 1.0, S0, _randn(9, *args[2].shape), None, F32)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_without_a_gate_is_a_gate_of_one(dtype, gated):
    *args, S0 = _inputs(3, 1, 400, 1, 2, 64, 64, dtype, gated=gated)
    o, S = K.fwd_delta(*args, initial_state=S0, return_state=True)
    _check_forward(args, _rows(1, 400), 1.0, S0, o, S, dtype)
    if not gated:
        same = K.fwd_delta(*args[:4], torch.zeros(1, 400, 2, device=DEV), initial_state=S0, return_state=True)
        assert torch.equal(o, same[0]) and torch.equal(S, same[1])


@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_beta_at_its_ends(dtype, beta):
    # beta 2 reflects (no contraction, still no growth); beta 0 writes nothing
    q, k, v, b, ld, S0 = _inputs(8, 1, 260, 2, 2, 64, 64, dtype)
    args = (q, k, v, torch.full_like(b, beta), ld)
    o, S = K.fwd_delta(*args, initial_state=S0, return_state=True)
    _check_forward(args, _rows(1, 260), 1.0, S0, o, S, dtype)
    _check_backward(args, _rows(1, 260), 1.0, S0, _randn(9, *v.shape, dtype=dtype), None, dtype)
    if beta == 0.0:
        assert not K.fwd_delta(*args).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_tokens_without_a_step(dtype):
    # padding by beta = 0: nothing is written there, and v has no gradient
    *args, S0 = _inputs(61, 1, 200, 1, 2, 64, 40, dtype)
    args[3][:, 50:90] = 0.0
    args[3][:, 128] = 0.0
    dO = _randn(9, *args[2].shape, dtype=dtype)
    _, _, dv, db, _, _ = _check_backward(args, _rows(1, 200), 1.0, S0, dO, None, dtype)
    assert not dv[:, 50:90].any() and not dv[:, 128].any() and dv[:, 49].any() and db[:, 50:90].any()
    # and steps of any size
    args[3][:, 50:90], args[3][:, 128] = 1e-12, 3e4
    args[1][:, 128] = 0.0
    _, S = K.fwd_delta(*args, initial_state=S0, return_state=True)
    _check_forward(args, _rows(1, 200), 1.0, S0, None, S, dtype)
    db = K.bwd_delta(*args[:4], dO, args[4], initial_state=S0)[3]
    assert torch.isfinite(db).all() and db[:, 50:90].any()


@pytest.mark.parametrize("at", [130, 511, 640, 999])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_non_finite_tokens_in_segments(dtype, at):
    *args, S0 = _inputs(62, 1, 1000, 2, 2, 64, 64, dtype)
    clean, cleanS = K.fwd_delta(*args, initial_state=S0, return_state=True)
    for which, value in (("v", float("nan")), ("v", float("inf")), ("k", float("nan")), ("beta", float("inf")), ("ld", float("nan"))):
        bad = [x.clone() for x in args]
        i = "q k v beta ld".split().index(which)
        bad[i][(0, at, 0) + ((5,) if i < 3 else ())] = value
        o, S = K.fwd_delta(*bad, initial_state=S0, return_state=True)
        assert torch.equal(o[:, :at], clean[:, :at]), which
        assert torch.equal(o[:, :, 1], clean[:, :, 1]) and torch.equal(S[:, 1], cleanS[:, 1]), which
        if which == "v":
            cols = [c for c in range(64) if c != 5]
            assert torch.isnan(o[0, at:, 0, 5]).all() and torch.isnan(S[0, 0, :, 5]).all()
            assert torch.equal(o[0, :, 0][:, cols], clean[0, :, 0][:, cols]) and torch.equal(S[0, 0][:, cols], cleanS[0, 0][:, cols])
        else:
            assert not torch.isfinite(o[0, at:, 0]).any() and not torch.isfinite(S[0, 0]).any(), which


def test_delta_keys_that_repeat():
    # one key over and over: the system is as far from the unit matrix as it gets
    q, k, v, b, ld, S0 = _inputs(12, 1, 200, 1, 1, 64, 64, F32, gated=False)
    args = (q, k[:, :1].expand(1, 200, 1, 64), v, torch.ones_like(b), None)
    o, S = K.fwd_delta(*args, return_state=True)
    _check_forward(args, _rows(1, 200), 1.0, None, o, S, F32)
    args = tuple(x.to(BF) for x in args[:4])
    _check_forward((*args, None), _rows(1, 200), 1.0, None, K.fwd_delta(*args), None, BF)


@pytest.mark.parametrize("ld", [-float("inf"), -1e30, -300.0, -40.0, 0.01])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_decays_of_any_strength(dtype, ld):
    # every third token forgets (or remembers more than there was)
    *args, S0 = _inputs(4, 1, 150, 1, 2, 64, 64, dtype)
    args[4][:, ::3] = ld
    o, S = K.fwd_delta(*args, initial_state=S0, return_state=True)
    _check_forward(args, _rows(1, 150), 1.0, S0, o, S, dtype)
    dO = _randn(5, 1, 150, 2, 64, dtype=dtype)
    grads = K.bwd_delta(*args[:4], dO, args[4], initial_state=S0)
    assert all(torch.isfinite(x).all() for x in grads)
    if ld < -200:
        assert not grads[4][:, ::3].any()            # a decay of zero has no gradient


@pytest.mark.parametrize("lengths", [[1], [0], [0, 0, 5, 0], [64, 64, 64], [1, 0, 77, 512, 130, 1, 63], [1500, 3, 0, 700],
                                     [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_packed(dtype, lengths):
    n, lead, tail = sum(lengths), 3, 70
    T = lead + n + tail
    *args, S0 = _inputs(n + 7, 1, T, 1, 2, 64, 40, dtype, N=len(lengths))
    cu = _cu(lengths, lead)
    rows = [(b, at + lead, m) for b, at, m in _rows(1, 0, lengths)]
    o, S = K.fwd_delta(*args, scale=0.5, initial_state=S0, return_state=True, cu_seqlens=cu)
    _check_forward(args, rows, 0.5, S0, o, S, dtype)
    assert not o[:, :lead].any() and not o[:, lead + n:].any()
    out = torch.full_like(args[2], 7.0)
    K.fwd_delta(*args, scale=0.5, initial_state=S0, cu_seqlens=cu, out=out)
    assert torch.all(out[:, :lead] == 7.0) and torch.all(out[:, lead + n:] == 7.0)
    _check_forward(args, rows, 0.5, S0, out, None, dtype)
    for i, m in enumerate(lengths):
        if m == 0:
            assert torch.equal(S[i], S0[i])
    dO, dS = _randn(4, *args[2].shape, dtype=dtype), _randn(5, *S0.shape)
    got = _check_backward(args, rows, 0.5, S0, dO, dS, dtype, cu=cu)
    for g in got[:5]:
        assert not g[:, :lead].any() and not g[:, lead + n:].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_rows_of_no_sequence_are_not_looked_at(dtype):
    lengths, lead, tail = [70, 0, 129, 64, 1], 5, 40
    T = lead + sum(lengths) + tail
    *args, S0 = _inputs(41, 1, T, 1, 2, 64, 64, dtype, N=len(lengths))
    dO, cu = _randn(4, *args[2].shape, dtype=dtype), _cu(lengths, lead)
    want = K.fwd_delta(*args, initial_state=S0, return_state=True, cu_seqlens=cu), K.bwd_delta(
        *args[:4], dO, args[4], initial_state=S0, cu_seqlens=cu)
    for x in (*args, dO):
        x[:, :lead] = float("nan")
        x[:, T - tail:] = float("inf")
    got = K.fwd_delta(*args, initial_state=S0, return_state=True, cu_seqlens=cu), K.bwd_delta(
        *args[:4], dO, args[4], initial_state=S0, cu_seqlens=cu)
    assert all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 64, 128), (BF, 40, 80), (BF, 128, 72), (F32, 32, 80), (F32, 64, 64)])
def test_delta_backward_of_more_chunks_than_workgroups(dtype, dk, dv):
    # 6 x 46 chunks: a workgroup of the gradients takes two, and value heads in turn; alone, a sequence's fit at once
    B, T = 6, 2900
    *args, S0 = _inputs(43, B, T, 1, 2, dk, dv, dtype)
    dO = _randn(4, B, T, 2, dv, dtype=dtype)
    got = K.bwd_delta(*args[:4], dO, args[4], initial_state=S0)
    for i in (0, 3, 5):
        one = K.bwd_delta(*[x[i:i + 1] for x in args[:4]], dO[i:i + 1], args[4][i:i + 1], initial_state=S0[i:i + 1])
        for name, x, y, t in zip("dq dk dv dbeta dlog dstate".split(), got, one, (dtype,) * 4 + (F32,) * 2):
            # both are off by what test_delta_errors_by_their_norm allows
            few = 2.0 ** -17 if dtype == BF else 2.0 ** -18
            tol = max(4 * U[BF], few) if t == BF else 2 * few * (16 if name == "dlog" else 2)
            err = (x[i:i + 1].double() - y.double()).norm() / y.double().norm()
            assert err <= tol, (name, float(err), tol)


def test_delta_packed_offsets_outside_the_rows_are_clamped():
    *args, S0 = _inputs(1, 1, 100, 1, 1, 64, 64, BF, N=2)
    bad = torch.tensor([-5, 1 << 30, 90], dtype=torch.int32, device=DEV)
    o, S = K.fwd_delta(*args, initial_state=S0, return_state=True, cu_seqlens=bad)
    K.bwd_delta(*args[:4], args[2], args[4], initial_state=S0, cu_seqlens=bad)
    torch.cuda.synchronize()
    assert torch.equal(o, K.fwd_delta(*args, initial_state=S0[:1], return_state=True)[0])
    assert torch.equal(S[1], S0[1])


def test_delta_packed_is_what_its_sequences_are_alone():
    lengths = [130, 64, 1, 333]
    *args, S0 = _inputs(2, 1, sum(lengths), 2, 4, 64, 64, BF, N=4)
    o, S = K.fwd_delta(*args, initial_state=S0, return_state=True, cu_seqlens=_cu(lengths))
    for i, (_, at, n) in enumerate(_rows(1, 0, lengths)):
        one = K.fwd_delta(*[x[:, at:at + n] for x in args], initial_state=S0[i:i + 1], return_state=True)
        if n <= 64:                                  # one chunk: in neither cut into segments
            assert torch.equal(o[:, at:at + n], one[0]) and torch.equal(S[i:i + 1], one[1])
        _check_forward([x[:, at:at + n] for x in args], _rows(1, n), 1.0, S0[i:i + 1], *one, BF)
    _check_forward(args, _rows(1, 0, lengths), 1.0, S0, o, S, BF)


def _check_backward(args, rows, scale, S0, dO, dS, dtype, cu=None):
    q, k, v, b, ld = args
    got = K.bwd_delta(q, k, v, b, dO, ld, scale=scale, initial_state=S0, dfinal_state=dS, cu_seqlens=cu)
    H, share, dk = v.shape[2], v.shape[2] // q.shape[2], q.shape[-1]
    want = {"dq": np.zeros(q.shape), "dk": np.zeros(q.shape)}
    tol = {"dq": np.zeros(q.shape), "dk": np.zeros(q.shape)}
    few = 2.0 ** -24 * (dk + v.shape[-1] + 256)
    for i, h, bb, s, (nq, nk, nv, nb, nl) in _heads(q, k, v, b, ld, rows):
        first, last = None if S0 is None else _np(S0)[i, h], None if dS is None else _np(dS)[i, h]
        G = _np(dO)[bb, s, h]
        ref = O.delta_backward(nq, nk, nv, nb, nl, G, scale, first, last)
        n = len(nq)
        M = O.delta_sizes(nq, nk, nv, nb, nl, first).max()
        # the recurrence in reversed time, where q dO is added
        R = max([np.linalg.norm(x, axis=0).max() for x in _reverse_states(nq, nk, nb, nl, G, scale, last)], default=0.0)
        R = R + np.abs(scale) * (np.linalg.norm(nq, axis=1).max() * np.abs(G).max() if n else 0.0)
        E = _step(n, dk, dtype) * 4
        if n:
            Bq, Bk, Bl = O.delta_gradient_sizes(nq, nk, nv, nb, nl, G, scale, first, last)
            u = 2 * U[BF] * 1.02 if dtype == BF else 0.0
            hk = h // share
            for name, r, B, size in (("dq", ref[0], Bq, M * np.abs(scale) * np.linalg.norm(G, axis=1, keepdims=True)),
                                     ("dk", ref[1], Bk, 2 * M * R * np.sqrt(v.shape[-1]))):
                want[name][bb, s, hk] += r
                tol[name][bb, s, hk] += (u + few) * B + E * size
            _inside(got[2][bb, s, h], ref[2], U[dtype] * 1.01 * np.abs(ref[2]) + E * R, f"dv {i} {h}")
            _inside(got[3][bb, s, h], ref[3], U[dtype] * 1.01 * np.abs(ref[3]) + E * R * M * np.sqrt(v.shape[-1]) * 2, f"dbeta {i} {h}")
            if ld is not None:
                w = 16 * (2.0 ** -18 if dtype == BF else 2.0 ** -24)
                _inside(got[4][bb, s, h], ref[4], (w + few) * Bl + E * R * M * np.sqrt(v.shape[-1] * dk) * 2, f"dlog_decay {i} {h}")
        if S0 is not None:
            _inside(got[5][i, h], ref[5], _step(n, dk, dtype) * R + 2.0 ** -24 * np.abs(ref[5]), f"dstate {i} {h}")
    for j, name in enumerate(("dq", "dk")):
        _inside(got[j], want[name], tol[name] + U[dtype] * 1.01 * np.abs(want[name]), name)
    assert ld is not None or got[4] is None
    return [x for x in got if x is not None]


def _reverse_states(q, k, b, ld, dO, scale, dS):
    D = np.zeros((q.shape[1], dO.shape[1])) if dS is None else dS.copy()
    out = [D]
    for t in range(len(q) - 1, -1, -1):
        D = D + scale * np.outer(q[t], dO[t])
        out.append(D)
        D = np.exp(ld[t]) * (D - b[t] * np.outer(k[t], k[t] @ D))
    return out + [D]


@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_backward(dtype, shape, states):
    B, T, Hk, H, dk, dv = shape
    *args, S0 = _inputs(sum(shape) + 1, *shape, dtype)
    dO = _randn(5, B, T, H, dv, dtype=dtype)
    _check_backward(args, _rows(B, T), 0.25, S0 if states else None, dO, _randn(6, *S0.shape) if states else None, dtype)


@pytest.mark.parametrize("shape", [(1, 1000, 1, 1, 64, 64), (1, 1000, 1, 2, 128, 128), (2, 200, 2, 2, 64, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_errors_by_their_norm(dtype, shape):
    # The bounds above add up what could go one way.  Roundings do not: by its 2-norm an output is off by the half
    # step of its own type, dq and dk by twice as much (factors rounded once), what stays in fp32 by a few steps of
    # the operands' terms (bf16 2^-18 each, for dlog_decay 2^-17 of terms that cancel by 2^4 here; fp32 64 steps).
    B, T, Hk, H, dk, dv = shape
    *args, S0 = _inputs(77, *shape, dtype)
    dO, dS = _randn(5, B, T, H, dv, dtype=dtype), _randn(6, *S0.shape)
    o, S = K.fwd_delta(*args, scale=0.25, initial_state=S0, return_state=True)
    got = K.bwd_delta(*args[:4], dO, args[4], scale=0.25, initial_state=S0, dfinal_state=dS)
    share = H // Hk
    want = [np.zeros(x.shape) for x in (o, S, *got)]
    for i, h, b, s, (q, k, v, be, ld) in _heads(*args, _rows(B, T)):
        want[0][b, s, h], want[1][i, h] = O.delta_recurrent(q, k, v, be, ld, 0.25, _np(S0)[i, h])
        g = O.delta_backward(q, k, v, be, ld, _np(dO)[b, s, h], 0.25, _np(S0)[i, h], _np(dS)[i, h])
        want[2][b, s, h // share] += g[0]
        want[3][b, s, h // share] += g[1]
        for j in (2, 3, 4):
            want[2 + j][b, s, h] = g[j]
        want[7][i, h] = g[5]
    few = 2.0 ** -17 if dtype == BF else 2.0 ** -18
    half = max(2.0 ** -8 if dtype == BF else 0.0, few)
    for name, x, r, tol in zip("o state dq dk dv dbeta dlog_decay dstate".split(), (o, S, *got), want,
                               (half, few, 2 * half, 2 * half, half, half, 16 * few, few)):
        err = np.linalg.norm(_np(x) - r) / np.linalg.norm(r)
        print(f"{name}: {err:.2e} of {tol:.2e}")
        assert err <= tol, name


def test_delta_backward_against_differences():
    # central differences of the forward pass itself, in fp32: off by rounding, 2^-22 of the loss's terms over the
    # step, and by the step squared
    q, k, v, b, ld, S0 = _inputs(21, 1, 70, 1, 2, 16, 16, F32)
    leaves = [q, k, v, b, ld, S0]
    dO, dS = _randn(6, 1, 70, 2, 16), _randn(7, 1, 2, 16, 16)

    def loss(q, k, v, b, ld, S0):
        o, S = K.fwd_delta(q, k, v, b, ld, initial_state=S0, return_state=True)
        return float((o.double() * dO).sum() + (S.double() * dS).sum()), float((o * dO).abs().sum() + (S * dS).abs().sum())

    grads = K.bwd_delta(q, k, v, b, dO, ld, initial_state=S0, dfinal_state=dS)
    for i, g in enumerate(grads):
        d = _randn(30 + i, *leaves[i].shape)
        h = 2.0 ** -8
        (hi, size), (lo, _) = (loss(*[x + s * h * d if j == i else x for j, x in enumerate(leaves)]) for s in (1, -1))
        want, got = (hi - lo) / (2 * h), float((g.double() * d).sum())
        assert abs(want - got) <= 2.0 ** -18 * size / h + h * h * 40 * size, (i, want, got)


def test_delta_many_sequences_and_segments_agree():
    # one long sequence alone is cut into segments, among others it is not
    *args, _ = _inputs(31, 8, 2000, 16, 16, 64, 64, BF)
    o, S = K.fwd_delta(*args, return_state=True)
    one = [x[:1, :, :1].contiguous() for x in args]
    a, s = K.fwd_delta(*one, return_state=True)
    _check_forward(one, _rows(1, 2000), 1.0, None, a, s, BF)
    _check_forward(one, _rows(1, 2000), 1.0, None, o[:1, :, :1], S[:1, :1], BF)
    dO = _randn(3, *args[2].shape, dtype=BF)
    _check_backward(one, _rows(1, 2000), 1.0, None, dO[:1, :, :1].contiguous(), None, BF)
    full, part = K.bwd_delta(*args[:4], dO, args[4]), K.bwd_delta(*one[:4], dO[:1, :, :1], one[4])
    for x, y in zip(full[:4], part[:4]):
        assert (x[:1, :, :1].float() - y.float()).norm() <= 2.0 ** -7 * y.float().norm()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_strides(dtype):
    B, T, H, d = 2, 150, 3, 64
    q, k, v, b, ld, S0 = _inputs(5, B, T, H, H, d, d, dtype)
    dO = _randn(6, B, T, H, d, dtype=dtype)
    ref = K.fwd_delta(q, k, v, b, ld, initial_state=S0, return_state=True)
    refg = K.bwd_delta(q, k, v, b, dO, ld, initial_state=S0)
    head_major = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v, dO)]
    fused = torch.cat([q, k, v, dO], -1)
    cut = [fused[..., i * d:(i + 1) * d] for i in range(4)]
    wide = torch.stack([b, b], -1)[..., 0], torch.stack([ld, ld], 2)[:, :, 1]
    for (q2, k2, v2, g2), (b2, l2) in ((head_major, (b, ld)), (cut, wide), ([q, k, v, dO], (b.transpose(1, 2).contiguous().transpose(1, 2), ld))):
        got = K.fwd_delta(q2, k2, v2, b2, l2, initial_state=S0, return_state=True)
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
        got = K.bwd_delta(q2, k2, v2, b2, g2, l2, initial_state=S0)
        assert all(torch.equal(x, y) for x, y in zip(got, refg))
    out = torch.zeros(B, T, H, 2 * d, dtype=dtype, device=DEV)[..., d:]
    assert K.fwd_delta(q, k, v, b, ld, initial_state=S0, out=out) is out and torch.equal(out, K.fwd_delta(q, k, v, b, ld, initial_state=S0))
    # broadcast axes
    kx, bx, lx = k[:, :, :1].expand(B, T, H, d), b[:, :1].expand(B, T, H), ld[:1].expand(B, T, H)
    same = K.fwd_delta(q, kx.contiguous(), v, bx.contiguous(), lx.contiguous())
    assert torch.equal(K.fwd_delta(q, kx, v, bx, lx), same)


@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (3, 2, 4, 64, 64), (2, 1, 3, 128, 128), (2, 2, 2, 40, 72), (1, 2, 2, 8, 8), (1, 1, 2, 16, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_decode(dtype, shape, T):
    B, Hk, H, dk, dv = shape
    *args, S0 = _inputs(sum(shape), B, T, Hk, H, dk, dv, dtype)
    for ld in (args[4], None):
        S = S0.clone()
        o = K.decode_delta(*args[:4], S, ld, scale=0.5)
        for i, h, b, s, (q, k, v, be, l) in _heads(*args[:4], ld, _rows(B, T)):
            ref, refS = O.delta_recurrent(q, k, v, be, l, 0.5, _np(S0)[i, h])
            M = O.delta_sizes(q, k, v, be, l, _np(S0)[i, h])
            few = T * (dk + 16) * 2.0 ** -23
            _inside(S[i, h], refS, few * M, f"state {i} {h}")
            _inside(o[b, s, h], ref, U[dtype] * 1.01 * np.abs(ref) + 0.5 * np.linalg.norm(q, axis=1, keepdims=True) * few * M, f"o {i} {h}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_decode_of_more_sequences_than_a_grid_axis_has(dtype):
    B = 65537
    q, k, v, b, ld, S0 = (x[:1].expand(B, *x.shape[1:]) for x in _inputs(2, 1, 1, 1, 1, 16, 16, dtype))
    S = S0.contiguous()
    o = K.decode_delta(q, k, v, b, S, ld)
    assert torch.equal(o, o[:1].expand_as(o)) and torch.equal(S, S[:1].expand_as(S))
    one = S0[:1].contiguous()
    assert torch.equal(K.decode_delta(q[:1], k[:1], v[:1], b[:1], one, ld[:1]), o[:1]) and torch.equal(one, S[:1])


@pytest.mark.parametrize("at", [0, 17, 63, 64, 100, 255])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_delta_non_finite_tokens_reach_no_earlier_row(dtype, value, at):
    *args, S0 = _inputs(6, 1, 300, 1, 2, 64, 64, dtype)
    clean = K.fwd_delta(*args, initial_state=S0)
    for which in ("q", "k", "v", "beta", "ld"):
        if which == "ld" and value == -float("inf"):
            continue                                 # a decay of zero, an ordinary value
        bad = [x.clone() for x in args]
        i = "q k v beta ld".split().index(which)
        place = (0, at, 0) + ((5,) if i < 3 else ())
        bad[i][place] = value
        o = K.fwd_delta(*bad, initial_state=S0)
        assert torch.equal(o[:, :at], clean[:, :at]), which
        if which == "q":
            assert not torch.isfinite(o[0, at, 0]).all()
            rows = [t for t in range(300) if t != at]
            assert torch.equal(o[:, rows], clean[:, rows])
        elif which == "v":                           # its own column alone
            assert torch.isnan(o[0, at:, 0, 5]).all()
            cols = [c for c in range(64) if c != 5]
            assert torch.equal(o[0, :, 0][:, cols], clean[0, :, 0][:, cols])
            assert torch.equal(o[:, :, 1], clean[:, :, 1])
        else:
            assert not torch.isfinite(o[0, at:, 0]).any(), which
        if which in ("beta", "ld"):
            assert torch.equal(o[:, :, 1], clean[:, :, 1])


def test_delta_non_finite_key_that_only_overflows():
    # keys so large that their products are infinite: rows before them are as without
    *args, _ = _inputs(7, 1, 130, 1, 1, 64, 64, F32)
    clean = K.fwd_delta(*args)
    args[1][0, 40:42] = 3e38
    o = K.fwd_delta(*args)
    assert torch.equal(o[:, :40], clean[:, :40])
    assert not torch.isfinite(o[:, 42:]).any()


def test_delta_states_continue_prompts_and_tokens():
    B, T, H, d = 2, 200, 2, 64
    *args, S0 = _inputs(3, B, T + 3, H, H, d, d, F32)
    o, S = K.fwd_delta(*args, initial_state=S0, return_state=True)
    a, S1 = K.fwd_delta(*[x[:, :77] for x in args], initial_state=S0, return_state=True)
    b, S2 = K.fwd_delta(*[x[:, 77:T] for x in args], initial_state=S1, return_state=True)
    c = [K.decode_delta(*[x[:, t:t + 1] for x in args[:4]], S2, args[4][:, t:t + 1]) for t in range(T, T + 3)]
    _check_forward(args, _rows(B, T + 3), 1.0, S0, torch.cat([a, b, *c], 1), S2, F32)
    _check_forward(args, _rows(B, T + 3), 1.0, S0, o, S, F32)


def test_delta_empty_tensors():
    for B, T, Hk, H in ((0, 5, 2, 2), (2, 0, 2, 2), (2, 5, 2, 0)):
        q, v = torch.zeros(B, T, Hk, 32, device=DEV), torch.zeros(B, T, H, 16, device=DEV)
        b, S0 = torch.zeros(B, T, H, device=DEV), _randn(1, B, H, 32, 16)
        o, S = K.fwd_delta(q, q, v, b, b, initial_state=S0, return_state=True)
        assert o.shape == v.shape and torch.equal(S, S0)
        dq, dk, dv, db, dl, d0 = K.bwd_delta(q, q, v, b, v, b, initial_state=S0, dfinal_state=S0)
        assert dq.shape == q.shape and not dq.any() and not dk.any() and dl.shape == b.shape and torch.equal(d0, S0)
        K.decode_delta(q, q, v, b, S0.clone(), b)
        assert not K.fwd_delta(q, q, v, b, return_state=True)[1].any()


def test_delta_large_offsets():
    # rows behind 2^31 elements
    base = torch.zeros(1, 40000, 1, 60000, dtype=BF, device=DEV)          # 2.4e9 elements
    q, k, v, b, ld, _ = _inputs(4, 1, 40000, 1, 1, 64, 64, BF)
    views = [base[..., i * 64:(i + 1) * 64] for i in range(3)]
    for x, y in zip(views, (q, k, v)):
        x.copy_(y)
    assert torch.equal(K.fwd_delta(*views, b, ld), K.fwd_delta(q, k, v, b, ld))


def test_delta_of_more_workgroups_than_a_grid_axis_has():
    # 65535 one-token sequences of 260 heads: over 2^32 work-items, which one grid axis cuts off
    n, H, d = 65535, 260, 8
    one = _inputs(3, 1, 1, H, H, d, d, BF)[:5]
    o = K.fwd_delta(*[x.expand(n, *x.shape[1:]) for x in one])
    assert torch.equal(o, K.fwd_delta(*one).expand_as(o))


def test_delta_workspace_of_the_caller_and_two_calls_at_once():
    *args, S0 = _inputs(9, 1, 1000, 2, 2, 64, 64, BF)
    dO = _randn(5, *args[2].shape, dtype=BF)
    want = K.fwd_delta(*args, initial_state=S0, return_state=True), K.bwd_delta(*args[:4], dO, args[4], initial_state=S0)
    sizes = [K.delta_workspace_size(*args[:4], args[4], backward=x) for x in (False, True)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
            got.append((K.fwd_delta(*args, initial_state=S0, return_state=True, workspace=ws[0]),
                        K.bwd_delta(*args[:4], dO, args[4], initial_state=S0, workspace=ws[1])))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for a, b in zip(g, want) for x, y in zip(a, b))


def test_delta_refusals():
    q, k, v, b, ld, _ = _inputs(1, 1, 8, 2, 2, 64, 64, BF)
    cu = _cu([8])
    with pytest.raises(TypeError):
        K.fwd_delta(q.half(), k.half(), v.half(), b.half())
    for bad in (lambda: K.fwd_delta(q, k[..., :32], v, b), lambda: K.fwd_delta(q, k, v.float(), b),
                lambda: K.fwd_delta(q, k, v, b.float()), lambda: K.fwd_delta(q, k, v, b[:, :4]),
                lambda: K.fwd_delta(q, k, v, b, ld.double()), lambda: K.fwd_delta(q, k, v, b, ld[..., :1]),
                lambda: K.fwd_delta(q, k, v, b, ld.cpu()), lambda: K.fwd_delta(q, k, v, b.cpu()),
                lambda: K.fwd_delta(q, k, v[:, :, :1], b[..., :1]), lambda: K.fwd_delta(q[:, :, :0], k[:, :, :0], v, b),
                lambda: K.fwd_delta(q, k, v, b, cu_seqlens=cu.long()), lambda: K.fwd_delta(q, k, v, b, cu_seqlens=cu[:1]),
                lambda: K.fwd_delta(*[x.expand(2, *x.shape[1:]) for x in (q, k, v, b)], cu_seqlens=cu),
                lambda: K.fwd_delta(q, k, v, b, initial_state=torch.zeros(1, 2, 64, 32, device=DEV)),
                lambda: K.fwd_delta(q, k, v, b, out=torch.empty_like(v, dtype=F32)),
                lambda: K.fwd_delta(q[..., ::2], k[..., ::2], v, b),
                lambda: K.bwd_delta(q, k, v, b, v.float()), lambda: K.bwd_delta(q, k, v, b, v[:, :4]),
                lambda: K.bwd_delta(q, k, v, b, v, dfinal_state=torch.zeros(2, 2, 64, 64, device=DEV)),
                lambda: K.decode_delta(q, k, v, b, torch.zeros(1, 2, 64, 64, device=DEV, dtype=BF)),
                lambda: K.decode_delta(q, k, v, b, None),
                lambda: K.parallel_delta_attn(q, k, v, b, ld, cu_seqlens=cu, rotary=K.rotary_rates(64)),
                lambda: K.parallel_delta_attn(q, k, v, b, ld, qk_norm="l1"),
                lambda: K.parallel_delta_attn(q, k, v, b, ld, norm=(torch.ones(32, device=DEV), None))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: K.fwd_delta(*[x[..., :12].contiguous() for x in (q, k, v)], b),                    # 24-byte rows
                lambda: K.fwd_delta(*[torch.zeros(1, 8, 2, 136, device=DEV, dtype=BF)] * 3, b),
                lambda: K.fwd_delta(q, k, v, b, scale=float("nan")),
                lambda: K.fwd_delta(q, k, v, b, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(K.KataError):
            bad()


# ---- norms of queries and keys, positions of several axes --------------------------------------------

QK = [(1, 1, 1, 1, 2, 2, False), (2, 3, 2, 1, 64, 64, False), (2, 50, 4, 2, 64, 64, True), (1, 17, 3, 3, 80, 48, False),
      (1, 9, 2, 1, 80, 46, True), (3, 5, 2, 2, 24, 22, False), (1, 40, 2, 2, 128, 128, False), (1, 6, 1, 1, 256, 256, True),
      (1, 6, 1, 1, 256, 250, True), (1, 6, 2, 1, 256, 2, False), (1, 7, 3, 1, 33, 0, False), (1, 700, 16, 16, 64, 64, False),
      (1, 3000, 2, 1, 40, 32, False)]


def _qk_tol(x, w, r, mag, dtype, ref):
    """Sums of squares and roots: 32 roundings; angles 2^-21 of both coordinates, at most the row's largest."""
    z = np.abs(x) * r * (1.0 if w is None else np.abs(w))
    return U[dtype] * 1.01 * np.abs(ref) + (2.0 ** -21 + 48 * 2.0 ** -24) * max(mag, 1.0) * 2 * z.max(-1, keepdims=True)


@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("B,T,H,Hk,D,rot,interleaved", QK)
@pytest.mark.parametrize("dtype,wtype", [(BF, F32), (BF, BF), (F32, F32), (F32, None)])
def test_qk_norm(dtype, wtype, B, T, H, Hk, D, rot, interleaved, l2, axes):
    q, k = 3 * _randn(1, B, T, H, D, dtype=dtype), _randn(2, B, T, Hk, D, dtype=dtype)
    wq, wk = (None, None) if wtype is None else ((_randn(3, D) * 0.2 + 1).to(wtype), (_randn(4, D) * 0.2 + 1).to(wtype))
    kw, angles, mag = dict(eps=1e-3, l2=l2), None, 1.0
    if rot:
        rates, mag = K.rotary_rates(rot)[0], 1.25
        pos = torch.randint(-5, 100000, (axes, B, T) if axes > 1 else (B, T), generator=torch.Generator().manual_seed(1)).to(DEV)
        which = torch.arange(rot // 2, dtype=torch.int32, device=DEV) % axes if axes > 1 else None
        kw.update(rates=rates, positions=pos, interleaved=interleaved, magnitude=mag, axes=which)
        at = _np(pos)[..., None] if axes == 1 else np.moveaxis(_np(pos)[_np(which).astype(int)], 0, -1)
        angles = at * _np(rates)
    got = K.fwd_qk_norm(q, k, wq, wk, **kw)
    dq, dk = _randn(5, *q.shape, dtype=dtype), _randn(6, *k.shape, dtype=dtype)
    grads = K.bwd_qk_norm(dq, dk, q, k, wq, wk, **kw)
    for i, (x, w, dy) in enumerate(((q, wq, dq), (k, wk, dk))):
        x, dy, w_ = _np(x), _np(dy), None if w is None else _np(w)
        n = 1 if l2 else D
        r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / n + 1e-3)
        ref = O.qk_norm(x, w_, 1e-3, l2, angles, interleaved, mag)
        _inside(got[i], ref, _qk_tol(x, w_, r, mag, dtype, ref), "y")
        dx, dw = O.qk_norm_backward(dy, x, w_, 1e-3, l2, angles, interleaved, mag)
        # t is a turned gradient; the second term has its sum over the row, of D terms
        t = 2 * np.abs(dy).max(-1, keepdims=True) * max(mag, 1.0) * (1.0 if w_ is None else np.abs(w_).max())
        size = r * t * (1 + r * r * np.abs(x) * np.abs(x).sum(-1, keepdims=True) / n)
        _inside(grads[i], dx, U[dtype] * 1.01 * np.abs(dx) + (2.0 ** -21 + (D + 64) * 2.0 ** -24) * size, "dx")
        if w is None:
            assert grads[2 + i] is None
        else:
            # sums over a lane's rows, the groups of a workgroup (64) and the workgroups (48 and 16)
            rows = B * T * (H if i == 0 else Hk)
            terms = (2 * np.abs(dy).max(-1, keepdims=True) * max(mag, 1.0) * np.abs(x) * r).sum((0, 1, 2))
            few = 2.0 ** -21 + (rows / 64 + 160) * 2.0 ** -24
            _inside(grads[2 + i], dw, U[w.dtype] * 1.01 * np.abs(dw) + few * terms, "dw")


def test_qk_norm_of_one_tensor_in_place_and_strides():
    B, T, H, D = 2, 30, 3, 64
    q, k, w = _randn(1, B, T, H, D, dtype=BF), _randn(2, B, T, 1, D, dtype=BF), _randn(3, D)
    rates = K.rotary_rates(D)[0]
    ref = K.fwd_qk_norm(q, k, w, w, rates=rates, offset=5)
    assert torch.equal(K.fwd_qk_norm(q, None, w, rates=rates, offset=5), ref[0])
    a, b = q.clone(), k.clone()
    got = K.fwd_qk_norm(a, b, w, w, rates=rates, offset=5, out=(a, b))
    assert got[0] is a and torch.equal(a, ref[0]) and torch.equal(b, ref[1])
    fused = torch.zeros(B, T, H, 2 * D + 3, dtype=BF, device=DEV)
    for lo in (0, 1, 8, D):                          # rows at any alignment
        x = fused[..., lo:lo + D]
        x.copy_(q)
        assert torch.equal(K.fwd_qk_norm(x, None, w, rates=rates, offset=5), ref[0])
        y = torch.zeros_like(fused)[..., lo:lo + D]
        assert torch.equal(K.fwd_qk_norm(q, None, w, rates=rates, offset=5, out=y), ref[0])
        dx, _, dw, _ = K.bwd_qk_norm(x, None, x, None, w, rates=rates)
        cx, _, cw, _ = K.bwd_qk_norm(q, None, q, None, w, rates=rates)
        assert torch.equal(dx, cx) and torch.equal(dw, cw)
    t = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(K.fwd_qk_norm(t, None, w, rates=rates, offset=5), ref[0])
    x = q[:1].expand(B, T, H, D)
    assert torch.equal(K.fwd_qk_norm(x, None, w), K.fwd_qk_norm(x.contiguous(), None, w))
    # without a turn: positions 0
    assert torch.equal(K.fwd_qk_norm(q, None, w), K.fwd_qk_norm(q, None, w, rates=rates, positions=torch.zeros(1, 1, dtype=torch.int32, device=DEV)))


def test_qk_norm_rows_of_zeros_infinities_and_nan():
    q = _randn(1, 1, 8, 2, 64, dtype=BF)
    clean = K.fwd_qk_norm(q, None)
    q[0, 1] = 0.0
    q[0, 3, 0, 5], q[0, 5, 1, 63] = float("inf"), float("nan")
    y = K.fwd_qk_norm(q, None)
    assert not y[0, 1].any()
    assert torch.isnan(y[0, 5, 1]).all()
    assert torch.isnan(y[0, 3, 0, 5]) and not y[0, 3, 0, :5].any()         # inf / inf, and the others over infinity
    keep = torch.ones(8, 2, dtype=torch.bool)
    keep[1], keep[3, 0], keep[5, 1] = False, False, False
    assert torch.equal(y[0][keep], clean[0][keep])
    dx, *_ = K.bwd_qk_norm(q, None, q, None)
    assert torch.isfinite(dx[0][keep]).all() and torch.isfinite(dx[0, 1]).all()


def test_qk_norm_empty_and_its_workspace():
    w = torch.ones(64, device=DEV)
    for B, T, H, Hk in ((0, 3, 2, 1), (2, 0, 2, 1), (2, 3, 0, 0), (2, 3, 2, 0)):
        q, k = torch.ones(B, T, H, 64, device=DEV), torch.ones(B, T, Hk, 64, device=DEV)
        y = K.fwd_qk_norm(q, k, w, w)
        g = K.bwd_qk_norm(q, k, q, k, w, w)
        assert y[0].shape == q.shape and y[1].shape == k.shape and g[2].shape == w.shape
        if not q.numel():
            assert not g[2].any()
        if not k.numel():
            assert not g[3].any()
    q = _randn(1, 1, 5000, 2, 64)
    n = K.qk_norm_workspace_size(q)
    ws = torch.full((n + 512,), 7, dtype=torch.uint8, device=DEV)
    a = K.bwd_qk_norm(q, None, q, None, w, workspace=ws[:n])
    assert torch.all(ws[n:] == 7) and torch.equal(a[2], K.bwd_qk_norm(q, None, q, None, w)[2])
    assert K.bwd_qk_norm(q, None, q, None, w, params=False)[2] is None


def test_qk_norm_refusals():
    q, k, w = _randn(1, 1, 4, 2, 64, dtype=BF), _randn(2, 1, 4, 1, 64, dtype=BF), torch.ones(64, device=DEV)
    rates, pos, ax = K.rotary_rates(64)[0], torch.zeros(3, 1, 4, dtype=torch.int64, device=DEV), K.rotary_axes((10, 11, 11))
    for bad in (lambda: K.fwd_qk_norm(q, k[:, :2]), lambda: K.fwd_qk_norm(q, k.float()), lambda: K.fwd_qk_norm(q, k, w[:32]),
                lambda: K.fwd_qk_norm(q, k, w, w.bfloat16()), lambda: K.fwd_qk_norm(q, None, w, w),
                lambda: K.fwd_qk_norm(q, k, w.cpu()), lambda: K.fwd_qk_norm(q[:, :, :0], k),
                lambda: K.fwd_qk_norm(q, k, rates=rates.float()), lambda: K.fwd_qk_norm(q, k, positions=pos[0]),
                lambda: K.fwd_qk_norm(q[..., :32], k[..., :32], rates=rates), lambda: K.fwd_qk_norm(q, k, out=q),
                lambda: K.fwd_qk_norm(q, k, rates=rates, positions=pos, axes=ax[:5]),
                lambda: K.fwd_qk_norm(q, k, rates=rates, positions=pos[0], axes=ax),
                lambda: K.fwd_qk_norm(q, k, rates=rates, axes=ax), lambda: K.fwd_qk_norm(q, k, rates=rates, positions=pos, axes=ax.long()),
                lambda: K.rotary(q, k, rates, axes=ax), lambda: K.rotary(q, k, rates, positions=pos, axes=ax.cpu()),
                lambda: K.rotary(q, k, rates, positions=pos[..., :3], axes=ax),
                lambda: K.bwd_qk_norm(q, None, q, k), lambda: K.bwd_qk_norm(q.float(), k, q, k),
                lambda: K.bwd_qk_norm(q, k, q, k, w, workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        K.fwd_qk_norm(q.half(), k.half())
    for bad in (lambda: K.fwd_qk_norm(q, k, eps=-1.0), lambda: K.fwd_qk_norm(torch.ones(1, 1, 1, 258, device=DEV), None),
                lambda: K.fwd_qk_norm(q.float(), k.float(), w.bfloat16()),
                lambda: K.bwd_qk_norm(q, k, q, k, w, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))):
        with pytest.raises(K.KataError):
            bad()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,T,H,Hk,D,rot,interleaved", [x for x in QK if x[5]])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rotary_of_several_axes(dtype, B, T, H, Hk, D, rot, interleaved, inverse):
    q, k = _randn(1, B, T, H, D, dtype=dtype), _randn(2, B, T, Hk, D, dtype=dtype)
    rates, n = K.rotary_rates(rot)[0], rot // 2
    which = K.rotary_axes((n - n // 3 - n // 2, n // 3, n // 2), interleaved=interleaved)
    pos = torch.randint(-9, 500000, (3, B, T), generator=torch.Generator().manual_seed(2)).to(DEV)
    kw = dict(positions=pos, axes=which, interleaved=interleaved, magnitude=1.25, inverse=inverse)
    got = K.rotary(q, k, rates, **kw)
    angles = np.moveaxis(_np(pos)[_np(which).astype(int)], 0, -1) * _np(rates)
    for x, y in zip((q, k), got):
        ref = O.turn(_np(x), angles, interleaved, 1.25, inverse)
        tol = U[dtype] * 1.01 * np.abs(ref) + 2.0 ** -20 * 1.25 * np.abs(_np(x)).max(-1, keepdims=True) + 0 * ref
        _inside(y, ref, tol, "rotary")
    # one axis for all pairs is the plain turn; an axis that is not there is the nearest one
    one = K.rotary(q, k, rates, positions=pos[1], interleaved=interleaved, magnitude=1.25, inverse=inverse)
    for fill in (1, None):
        w = torch.full_like(which, 1) if fill else torch.full_like(which, 9)
        p = pos if fill else pos[:2]
        assert all(torch.equal(x, y) for x, y in zip(one, K.rotary(q, k, rates, **{**kw, "axes": w, "positions": p})))
    same = K.rotary(q, k, rates, **{**kw, "positions": pos[:, :1, :1].int().expand(3, B, T)})
    assert all(torch.equal(x, y) for x, y in zip(same, K.rotary(q, k, rates, **{**kw, "positions": pos[:, :1, :1]})))


# ---- a run of them together --------------------------------------------------------------------------

def _layer_inputs(T=130, dtype=F32):
    B, Hk, H, d = 1, 2, 4, 16
    return ([_randn(1, B, T, Hk, d, dtype=dtype), _randn(2, B, T, Hk, d, dtype=dtype), _randn(3, B, T, H, d, dtype=dtype),
             torch.sigmoid(_randn(4, B, T, H)).to(dtype), -0.1 * torch.rand(B, T, H).to(DEV), _randn(5, B, H, d, d),
             _randn(6, d) * 0.1 + 1, (_randn(7, d) * 0.1 + 1) / 5, _randn(8, d) * 0.1 + 1, _randn(9, d) * 0.1],
            torch.stack([torch.arange(T, device=DEV) // 9, torch.arange(T, device=DEV) % 9])[:, None])


@pytest.mark.parametrize("packed", [False, True])
def test_autograd_of_a_layer(packed):
    leaves, pos = _layer_inputs()
    leaves = [x.clone().requires_grad_() for x in leaves]
    q, k, v, b, ld, S0, wq, wk, w, bias = leaves
    T, H, d = 130, 4, 16
    lengths = [50, 0, 80] if packed else [T]
    if packed:
        S0 = _randn(10, 3, H, d, d).requires_grad_()
        leaves[5] = S0
    rates, mag = K.rotary_rates(d)
    which = K.rotary_axes((3, 5))
    y, S = K.parallel_delta_attn(q, k, v, b, ld, scale=0.5, initial_state=S0, return_state=True,
                                 cu_seqlens=_cu(lengths) if packed else None, qk_norm=(wq, wk, 1e-3),
                                 rotary=(rates, mag, which), positions=pos, interleaved=True, norm=(w, bias))
    g, gS = _randn(20, *y.shape), _randn(21, *S.shape)
    got = torch.autograd.grad((y * g).sum() + (S * gS).sum(), leaves)

    ref = [x.detach().double().cpu().requires_grad_() for x in leaves]
    rq, rk, rv, rb, rl, rS, rwq, rwk, rw, rbias = ref
    angle = pos.cpu().double()[which.cpu().long()].movedim(0, -1)[..., None, :] * rates.cpu()

    def normed(x, w):
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-3) * w
        a, c = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * angle.cos() - c * angle.sin(), a * angle.sin() + c * angle.cos()], -1).flatten(-2)

    tq, tk = (normed(x, w_)[0].repeat_interleave(2, 1) for x, w_ in ((rq, rwq), (rk, rwk)))
    loss, at = 0.0, 0
    for i, n in enumerate(lengths):
        s = rS[i]
        for t in range(at, at + n):
            s = torch.exp(rl[0, t])[:, None, None] * s
            u = rb[0, t][:, None] * (rv[0, t] - (tk[t][:, :, None] * s).sum(1))
            s = s + tk[t][:, :, None] * u[:, None]
            o = torch.nn.functional.layer_norm(0.5 * (tq[t][:, :, None] * s).sum(1), (d,), rw, rbias)
            loss = loss + (o * g[0, t].cpu().double()).sum()
        at += n
        loss = loss + (s * gS[i].cpu().double()).sum()
    for name, x, r in zip("q k v b ld S0 wq wk w bias".split(), got, torch.autograd.grad(loss, ref)):
        # a chain of fp32 operators on keys of length 4 / 5 (d = 16), a contraction: each is off by a few hundred
        # roundings of its largest entry.  (Keys of length 4 would grow by 4e26 along the 130 tokens, the largest
        # norm of the products of I - b k k^T: no digit of the gradient would be left, in any order of sums.)
        _inside(x, r.numpy(), 2048 * 2.0 ** -24 * float(r.abs().max()), name)


def test_autograd_of_the_norm_of_one_tensor():
    x, w = _randn(1, 2, 30, 3, 64).requires_grad_(), _randn(2, 64).requires_grad_()
    g, rates = _randn(3, 2, 30, 3, 64), K.rotary_rates(64)[0]
    got = torch.autograd.grad(K.qk_norm(x, None, w, rates=rates, offset=3), (x, w), g)
    want = K.bwd_qk_norm(g, None, x.detach(), None, w.detach(), rates=rates, offset=3)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[2])


def test_a_captured_training_step_of_the_layer():
    q, k, v, b, ld, _ = _inputs(51, 2, 700, 1, 2, 64, 64, BF)
    w, g, rates = _randn(6, 64), _randn(5, *v.shape, dtype=BF), K.rotary_rates(64)

    def step():
        leaves = [x.detach().requires_grad_() for x in (q, k, v, b, ld, w)]
        o = K.parallel_delta_attn(*leaves[:5], qk_norm="l2", rotary=rates, norm=(leaves[5], None))
        return (o, *torch.autograd.grad(o, leaves, g))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        for j, x in enumerate((q, k, v, g)):
            x.copy_(_randn(60 + 4 * i + j, *x.shape, dtype=BF))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.detach().clone() for x in out]
        want = step()
        assert all(torch.isfinite(x).all() for x in want)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_one_layer_prompt_then_tokens():
    B, T, Hk, H, d = 2, 150, 2, 4, 64
    q, k, v, b, ld, _ = _inputs(13, B, T + 4, Hk, H, d, d, F32)
    rates = K.rotary_rates(d)[0]
    full = K.parallel_delta_attn(q, k, v, b, ld, qk_norm="l2", rotary=(rates, 1.0))
    o, S = K.parallel_delta_attn(*[x[:, :T] for x in (q, k, v, b, ld)], qk_norm="l2", rotary=(rates, 1.0), return_state=True)
    outs = [o]
    for t in range(T, T + 4):
        one = slice(t, t + 1)
        a, c = K.fwd_qk_norm(q[:, one], k[:, one], l2=True, rates=rates, offset=t)
        outs.append(K.decode_delta(a, c, v[:, one], b[:, one], S, ld[:, one]))
    # both are off by some steps of fp32 of a state of size M at most
    M = float(v.abs().max()) * 40
    assert (torch.cat(outs, 1) - full).abs().max() <= 8 * _step(T, d, F32) * M


def test_the_layer_is_its_parts():
    (q, k, v, b, ld, S0, wq, wk, w, bias), pos = _layer_inputs(dtype=BF)
    rates, mag = K.rotary_rates(16, scaling="parts", factor=4.0, original_length=64)
    which = K.rotary_axes((4, 4))
    a, c = K.fwd_qk_norm(q, k, wq, wk, eps=1e-6, rates=rates, positions=pos, axes=which, magnitude=mag)
    o = K.fwd_delta(a, c, v, b, ld, scale=0.25, initial_state=S0)
    y = K.fwd_layer_norm(o, w, bias)
    assert torch.equal(y, K.parallel_delta_attn(q, k, v, b, ld, scale=0.25, initial_state=S0, qk_norm=(wq, wk),
                                                rotary=(rates, mag, which), positions=pos, norm=(w, bias)))
    a, c = K.rotary(q, k, rates, positions=pos, axes=which, magnitude=mag)
    assert torch.equal(K.fwd_delta(a, c, v, b, ld), K.parallel_delta_attn(q, k, v, b, ld, rotary=(rates, mag, which), positions=pos))
    # the other layers take positions of several axes, too
    kk, vv = k.repeat_interleave(2, 2), v
    qq, dec = q.repeat_interleave(2, 2), torch.full((4,), -0.1, device=DEV)
    a, c = K.rotary(qq, kk, rates, positions=pos, axes=which, magnitude=mag)
    assert torch.equal(K.fwd_decay(a, c, vv, dec), K.parallel_decay_attn(qq, kk, vv, dec, rotary=(rates, mag, which), positions=pos))
    x = [t[:, :128] for t in (qq, kk, vv)]
    a, c = K.rotary(x[0], x[1], rates, positions=pos[..., :128], axes=which, magnitude=mag)
    assert torch.equal(K.parallel_kata_attn(a, c, x[2]), K.parallel_kata_attn(*x, rotary=(rates, mag, which), positions=pos[..., :128]))


def test_gradients_of_broadcast_inputs_and_unused_outputs():
    B, T, H, d = 1, 70, 4, 32
    q, k, v, b, ld, S0 = _inputs(14, B, T, H, H, d, d, F32)
    kl, bl, ll = k[:, :, :1].clone().requires_grad_(), b[:, :1].clone().requires_grad_(), ld[..., :1].clone().requires_grad_()
    wide = kl.expand(B, T, H, d), bl.expand(B, T, H), ll.expand(B, T, H)
    o, S = K.parallel_delta_attn(q, wide[0], v, wide[1], wide[2], return_state=True)
    got = torch.autograd.grad(o.sum(), (kl, bl, ll), retain_graph=True)      # dO is a broadcast one
    want = K.bwd_delta(q, wide[0], v, wide[1], torch.ones_like(v), wide[2])
    assert torch.equal(got[0], want[1].sum(2, keepdim=True)) and torch.equal(got[1], want[3].sum(1, keepdim=True))
    assert torch.equal(got[2], want[4].sum(2, keepdim=True))
    sk, = torch.autograd.grad(S.sum(), kl)                                   # only the state is used
    want = K.bwd_delta(q, wide[0], v, wide[1], torch.zeros_like(v), wide[2], dfinal_state=torch.ones_like(S))
    assert torch.equal(sk, want[1].sum(2, keepdim=True))
    # shared heads: the sum over the value heads of each
    few = K.bwd_delta(q[:, :, :2], k[:, :, :2], v, b, v, ld)
    many = K.bwd_delta(q[:, :, :2].repeat_interleave(2, 2), k[:, :, :2].repeat_interleave(2, 2), v, b, v, ld)
    for x, y in zip(few[:2], many[:2]):
        y = y.view(B, T, 2, 2, d)
        assert (x - y.sum(3)).abs().max() <= 64 * 2.0 ** -24 * y.abs().max()
    assert torch.equal(few[2], many[2]) and torch.equal(few[4], many[4])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_that_arrive_at_any_alignment(dtype):
    q, k, v, b, ld, S0 = _inputs(15, 1, 70, 2, 2, 64, 64, dtype)
    lead, c, cs = torch.zeros(1, dtype=dtype, device=DEV), _randn(5, 1 + v.numel(), dtype=dtype), _randn(6, 1 + S0.numel())
    leaves = [x.clone().requires_grad_() for x in (q, k, v, b, ld, S0)]
    o, S = K.parallel_delta_attn(*leaves[:5], initial_state=leaves[5], return_state=True)
    loss = (torch.cat([lead, o.flatten()]) * c).sum() + (torch.cat([lead.float(), S.flatten()]) * cs).sum()
    got = torch.autograd.grad(loss, leaves)
    want = K.bwd_delta(q, k, v, b, c[1:].clone().view_as(v), ld, initial_state=S0, dfinal_state=cs[1:].clone().view_as(S0))
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_layer_of_an_empty_batch():
    for B, T in ((0, 5), (2, 0)):
        q = torch.empty(B, T, 2, 32, device=DEV, requires_grad=True)
        b = torch.empty(B, T, 2, device=DEV, requires_grad=True)
        w = torch.ones(32, device=DEV, requires_grad=True)
        o = K.parallel_delta_attn(q, q, q, b, b, qk_norm=(w, w), rotary=K.rotary_rates(32), norm=(w, w))
        grads = torch.autograd.grad(o.sum(), (q, b, w))
        assert o.shape == q.shape and grads[0].shape == q.shape and not grads[2].any()


def test_tensors_written_in_place_tell_autograd():
    q, k, v, b, ld, S = _inputs(16, 2, 3, 2, 2, 64, 64, F32)
    o, a, c = (torch.empty_like(q) for _ in range(3))
    for call, written in ((lambda: K.decode_delta(q, k, v, b, S, ld), [S]),
                          (lambda: K.decode_delta(q, k, v, b, S, ld, out=o), [S, o]),
                          (lambda: K.fwd_delta(q, k, v, b, ld, out=o), [o]),
                          (lambda: K.fwd_qk_norm(q, k, out=(a, c)), [a, c]),
                          (lambda: K.fwd_qk_norm(q, None, out=a), [a])):
        reads, before = [x._version for x in (q, k, v, b, ld)], [x._version for x in written]
        call()
        assert all(x._version > n for x, n in zip(written, before))
        assert reads == [x._version for x in (q, k, v, b, ld)]
    leaf = q.clone().requires_grad_()
    loss = K.parallel_delta_attn(leaf, k, v, b, ld, initial_state=S).sum()
    K.decode_delta(q, k, v, b, S, ld)                # a state that a backward pass still needs
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    with torch.inference_mode():
        s = S.clone()
        K.decode_delta(q, k, v, b, s, ld, out=torch.empty_like(v))
        K.fwd_qk_norm(q, k, out=(torch.empty_like(q), torch.empty_like(k)))


def test_timing_records_every_kernel():
    q, k, v, b, ld, _ = _inputs(17, 1, 900, 2, 2, 64, 64, BF)
    rates = K.rotary_rates(64)[0]
    K.fwd_delta(q, k, v, b, ld)
    K.timing_begin()
    a, c = K.fwd_qk_norm(q, k, l2=True, rates=rates)
    K.fwd_delta(a, c, v, b, ld)
    K.bwd_delta(a, c, v, b, v, ld)
    K.bwd_qk_norm(a, c, q, k, l2=True, rates=rates)
    K.decode_delta(q[:, :1], k[:, :1], v[:, :1], b[:, :1], torch.zeros(1, 2, 64, 64, device=DEV), ld[:, :1])
    t = K.timing_end()
    assert t["norm"][0] == 2 and t["chunk_output"][0] == 1 and t["bwd"][0] == 1 and t["decode"][0] == 1 and t["chunk_state"][0] == 2
    assert all(ms > 0 for n, ms in t.values() if n)


def test_side_stream():
    s = torch.cuda.Stream()
    q, k, v, b, ld, _ = _inputs(18, 1, 1000, 2, 2, 64, 64, BF)
    run = lambda: K.parallel_delta_attn(q, k, v, b, ld, qk_norm="l2", rotary=K.rotary_rates(64), norm=(None, None))  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("l2", [False, True])
def test_replays_of_captured_graphs(l2):
    # graphs of a training step and of a decode step, replayed in turn with eager work between
    q, k, v, b, ld, _ = _inputs(19, 1, 900, 1, 2, 64, 64, BF)
    g, w = _randn(5, *v.shape, dtype=BF), _randn(6, 64)
    if l2:
        w = w / w.abs().max()
    rates = K.rotary_rates(64)[0]
    tok = _inputs(20, 3, 1, 2, 2, 64, 64, BF)
    st = tok[5]

    def train():
        a, c = K.fwd_qk_norm(q, k, w, w, l2=l2, rates=rates)
        o, S = K.fwd_delta(a, c, v, b, ld, return_state=True)
        dq, dk, dv, db, dl, _ = K.bwd_delta(a, c, v, b, g, ld)
        return (o, S, dv, db, dl, *K.bwd_qk_norm(dq, dk, q, k, w, w, l2=l2, rates=rates))

    def same(x, y):                                  # bit by bit: keys of length 8 end in infinities and nan
        bits = torch.int16 if x.dtype == BF else torch.int32
        return torch.equal(x.contiguous().view(bits), y.contiguous().view(bits))

    def step():
        a, c = K.fwd_qk_norm(tok[0], tok[1], l2=True, rates=rates, offset=5)
        return K.decode_delta(a, c, *tok[2:4], st, tok[4])

    train(), K.decode_delta(*tok[:4], st.clone(), tok[4])
    torch.cuda.synchronize()
    graphs, outs, S0 = [], [], st.clone()
    for f in (train, step):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = f()
        graphs.append(gr), outs.append(out)
    st.copy_(S0)
    ref = S0.clone()
    for i in range(4):
        for j, x in enumerate((q, k, v, g)):
            x.copy_(_randn(30 + 4 * i + j, *x.shape, dtype=BF))
        k.mul_(0.1)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs[0]], outs[1].clone(), st.clone()
        want = train()
        assert all(same(x, y) for x, y in zip(got[0], want))
        assert not l2 or all(torch.isfinite(x).all() for x in want)
        st.copy_(ref)
        y = step()
        assert torch.equal(got[1], y) and torch.equal(got[2], st)
        ref = st.clone()
