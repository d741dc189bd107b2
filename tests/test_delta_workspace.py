"""The sizes that include/kata.h gives for the gated delta rule's workspaces, against what the library asks for (no GPU)."""

import ctypes

import pytest

import kernelized_psd_feature_amd as K
from kernelized_psd_feature_amd import delta as KD


def _bytes(backward, **fields):
    pr = KD._DeltaProblem()
    for name, x in fields.items():
        setattr(pr, name, x)
    pr.scale = 1.0
    T, Hk, H, dk, dv = pr.T, pr.Hk, pr.H, pr.dk, pr.dv
    for s, h, w in ((pr.sq, Hk, dk), (pr.sk, Hk, dk), (pr.sv, H, dv), (pr.so, H, dv), (pr.sdo, H, dv), (pr.sbeta, H, 1), (pr.sdecay, H, 1)):
        s[:] = (T * h * w, h * w, w)
    size = K._lib().kata_bwd_delta_workspace_size if backward else K._lib().kata_fwd_delta_workspace_size
    return size(ctypes.byref(pr))


@pytest.mark.parametrize("dtype,dk,dv,rows,columns", [(1, 64, 64, 64, 64), (1, 24, 40, 64, 48), (1, 128, 72, 128, 80), (0, 32, 64, 32, 64),
                                                      (0, 36, 100, 64, 112), (0, 68, 4, 128, 16)])
def test_workspaces_are_what_the_header_says(dtype, dk, dv, rows, columns):
    n, H, chunks = 512, 8, 4                         # whole sequences: no segments
    fields = dict(n_seq=n, H=H, Hk=H, T=64 * chunks - 5, dk=dk, dv=dv, packed=0, dtype=dtype)
    kept = n * H * chunks * (5 * 64 + 10 * 256) * 4
    assert _bytes(False, **fields) == kept
    assert _bytes(True, **fields) == kept + n * H * (2 * chunks * (rows + 64) * columns + rows * columns) * 4
    # few chunks and shared heads of q and k: their gradients by value heads, and segments
    few = dict(fields, n_seq=1, Hk=1)
    kept = H * chunks * (5 * 64 + 10 * 256) * 4
    want = kept + H * (2 * chunks * (rows + 64) * columns + rows * columns) * 4 + 2 * (64 * chunks - 5) * H * dk * 4
    assert want <= _bytes(True, **few) < want + 16 * 256       # (parts begin at multiples of 256 bytes)
