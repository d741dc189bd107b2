"""Bounds by the 2-norm for the gated delta rule's outputs and gradients, one for each sequence, head and output; used by
test_gpu_delta_norms.py, and by test_delta_norms.py, which shows that they reject a gradient without one of its terms.

An output is off by its own rounding, at most half a step of its type (bf16 2^-8 of it, fp32 2^-24), and by its factors'
roundings: each is a product of two numbers that come out of fp32 sums, kept in two bf16 terms (2^-18 each, 2^-17 of the product), or
in fp32, where the sums of up to 128 + 64 terms leave about 8 half steps, sqrt(192 / 3), of 2^-24 (2^-21).  They are relative to
the factors' norms at the token (oracle.delta_token_sizes), and there are at most eight of them on the way of a chunk (the state, its
gradient, the inverse, the correction before and after it, the scores, their gradient, the sum); with keys of unit length
what comes from earlier chunks fades."""

import numpy as np
import torch

from oracle import delta_oracle as O

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TERMS = {BF: 8 * 2.0 ** -17, F32: 8 * 2.0 ** -21}
IN_FP32 = ("dld", "state", "dS0")                    # whatever the inputs' type
GRADIENTS = "dq dk dv db dld dS0".split()

# B, T, Hk, H, dk, dv
SHAPES = [(1, 1, 1, 1, 64, 64), (2, 2, 1, 2, 64, 64), (1, 63, 1, 1, 32, 32), (1, 64, 2, 2, 64, 64), (2, 65, 1, 3, 64, 64),
          (1, 130, 1, 1, 16, 8), (1, 200, 2, 2, 128, 128), (1, 200, 1, 2, 64, 128), (1, 200, 1, 1, 128, 40), (1, 300, 3, 3, 24, 72),
          (2, 700, 1, 1, 40, 104), (1, 1000, 2, 2, 64, 64), (1, 1000, 1, 1, 128, 128), (1, 500, 1, 5, 8, 24), (2, 321, 2, 4, 96, 56)]
PACKED = [[1], [0, 0, 5, 0], [64, 64, 64], [1, 0, 77, 512, 130, 1, 63], [900, 3, 0, 400], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10]]


def randn(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def inputs(seed, B, T, Hk, H, dk, dv, dtype, n=None):
    """q, k, v, beta, log_decay, dO, S0, dS on the CPU: keys a little short of unit length, memories of one token to some
    hundred by head (the first one's reach over a chunk)."""
    k = randn(seed + 1, B, T, Hk, dk)
    window = 2.0 ** -torch.tensor([(5, 0, 8, 2, 6)[h % 5] for h in range(H)], dtype=F32)
    ld = -window * torch.rand(B, T, H, generator=torch.Generator().manual_seed(seed + 4))
    return [randn(seed, B, T, Hk, dk, dtype=dtype), (k * (0.99 / k.norm(dim=-1, keepdim=True))).to(dtype),
            randn(seed + 2, B, T, H, dv, dtype=dtype), torch.sigmoid(randn(seed + 3, B, T, H)).to(dtype), ld,
            randn(seed + 5, B, T, H, dv, dtype=dtype), randn(seed + 6, n or B, H, dk, dv), randn(seed + 7, n or B, H, dk, dv)]


def rows(B, T, lengths=None, first=0):
    """(batch row, first row, length) of the sequences."""
    if lengths is None:
        return [(i, 0, T) for i in range(B)]
    cu = first + np.concatenate([[0], np.cumsum(lengths)]).astype(int)
    return [(0, int(cu[i]), int(m)) for i, m in enumerate(lengths)]


def _np(x):
    return None if x is None else x.detach().to(torch.float64).cpu().numpy()


def heads(args, seqs, scale):
    """(sequence, head, head of q and k, batch row, rows, the oracle's arguments)."""
    q, k, v, b, ld, dO, S0, dS = (_np(x) for x in args)
    share = v.shape[2] // q.shape[2]
    for i, (bb, at, m) in enumerate(seqs):
        s = slice(at, at + m)
        for h in range(v.shape[2]):
            yield i, h, h // share, bb, s, (q[bb, s, h // share], k[bb, s, h // share], v[bb, s, h], b[bb, s, h],
                                            np.zeros(m) if ld is None else ld[bb, s, h], dO[bb, s, h], scale,
                                            None if S0 is None else S0[i, h], None if dS is None else dS[i, h])


def expected(args, seqs, scale, backward=O.delta_backward, forward=True, sizes=O.delta_token_sizes):
    """{(output, sequence, head): [reference, sizes]}; those of dq and dk are sums over the heads that share them."""
    want = {}

    def add(name, i, h, ref, size):
        old = want.get((name, i, h))
        want[name, i, h] = [ref, np.asarray(size)] if old is None else [old[0] + ref, old[1] + size]

    for i, h, hk, _, _, a in heads(args, seqs, scale):
        size = sizes(*a)
        if forward:
            o, S = O.delta_recurrent(*a[:5], a[6], a[7])
            add("o", i, h, o, size["o"]), add("state", i, h, S, size["state"])
        for name, g in zip(GRADIENTS, backward(*a)):
            add(name, i, hk if name in ("dq", "dk") else h, g, size[name])
    return want


def results(args, seqs, got):
    """The same keys' values of what the calls returned: {output: tensor}, and (B, T, heads ...) rows cut into sequences."""
    out = {}
    for name, x in got.items():
        if x is None:
            continue
        x = _np(x)
        for i, (bb, at, m) in enumerate(seqs):
            for h in range(x.shape[1 if name in ("state", "dS0") else 2]):
                out[name, i, h] = x[i, h] if name in ("state", "dS0") else x[bb, at:at + m, h]
    return out


def share_of_bound(got, ref, size, name, dtype):
    """|got - ref| by norm over the bound; at most 1 is right, nan is not."""
    if not ref.size:
        return 0.0
    half = HALF[F32 if name in IN_FP32 else dtype]
    # below 2^-126 fp32 (and bf16) numbers lose digits, and may be zeros
    bound = half * np.linalg.norm(ref) + TERMS[dtype] * np.linalg.norm(size) + 2.0 ** -126 * ref.size ** 0.5
    err = np.linalg.norm(got - ref)
    return err / bound


def check(args, seqs, got, scale, dtype):
    """Every output in `got`, {name: tensor}; returns the worst share of a bound by output."""
    want, have, worst = expected(args, seqs, scale, forward="o" in got or "state" in got), results(args, seqs, got), {}
    bad = []
    for key, x in have.items():
        ref, size = want[key]
        share = share_of_bound(x, ref, size, key[0], dtype)
        worst[key[0]] = max(worst.get(key[0], 0.0), share)
        if not share <= 1.0:
            bad.append((key, float(share)))
    print("shares of the bounds:", {n: round(float(s), 3) for n, s in worst.items()}, flush=True)
    assert not bad, sorted(bad, key=lambda x: -x[1])[:8]
    return worst
