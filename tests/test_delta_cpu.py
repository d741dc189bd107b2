"""The gated delta rule, the norm of queries and keys and positions of several axes without a GPU: the C
ABI's refusals (fake, never dereferenced pointers: validation runs before any device call), the binding's
refusals, and the planner under the host sanitizers."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import kernelized_psd_feature_amd as K
from kernelized_psd_feature_amd import delta as KD
from kernelized_psd_feature_amd import layer as KL

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kernelized_psd_feature_amd", "csrc")
OK, INVALID, UNSUPPORTED, WORKSPACE, DEVICE = 0, 1, 2, 3, 4
FAKE = 0x7F0000000000


def _fake(n):
    return [ctypes.c_void_p(FAKE + i * (1 << 32)) for i in range(n)]


def _off(n):
    return ctypes.c_void_p(FAKE + n)


def _delta(n_seq=2, H=4, Hk=2, T=640, dk=64, dv=64, packed=0, dtype=1, scale=1.0):
    pr = KD._DeltaProblem()
    for name, x in dict(n_seq=n_seq, H=H, Hk=Hk, T=T, dk=dk, dv=dv, packed=packed, dtype=dtype, scale=scale).items():
        setattr(pr, name, x)
    for s, h, w in ((pr.sq, Hk, dk), (pr.sk, Hk, dk), (pr.sv, H, dv), (pr.so, H, dv), (pr.sdo, H, dv), (pr.sbeta, H, 1),
                    (pr.sdecay, H, 1)):
        s[:] = (T * h * w, h * w, w)
    return pr


NAMES = ("q", "k", "v", "beta", "ld", "cu", "s0", "o", "sT")


def _fwd(pr, ws=True, ws_bytes=None, **swap):
    lib = K._lib()
    a = dict(zip(NAMES, _fake(9)))
    a.update(swap)
    need = lib.kata_fwd_delta_workspace_size(ctypes.byref(pr)) if pr is not None else 0
    return lib.kata_fwd_delta(ctypes.byref(pr) if pr is not None else None, *a.values(), _fake(10)[9] if ws else None,
                              need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("field,value,code", [
    ("n_seq", 0, INVALID), ("H", 0, INVALID), ("Hk", 0, INVALID), ("Hk", 3, INVALID), ("T", 0, INVALID),
    ("dk", 0, INVALID), ("dv", -8, INVALID), ("dk", 12, UNSUPPORTED), ("dv", 136, UNSUPPORTED),
    ("T", (1 << 26) + 1, UNSUPPORTED), ("n_seq", 65536, UNSUPPORTED), ("dtype", 2, INVALID), ("packed", 2, INVALID),
    ("scale", float("nan"), INVALID), ("scale", float("inf"), INVALID),
])
def test_delta_refuses_bad_problems(field, value, code):
    pr = _delta()
    setattr(pr, field, value)
    assert _fwd(pr) == code
    assert K._lib().kata_last_error()
    assert K._lib().kata_fwd_delta_workspace_size(ctypes.byref(pr)) == 0


def test_delta_refuses_bad_pointers_strides_and_workspaces():
    assert _fwd(None) == INVALID
    for name in ("q", "k", "v", "beta", "o"):
        assert _fwd(_delta(), **{name: None}) == INVALID
    for name in ("q", "k", "v", "o", "s0", "sT"):
        assert _fwd(_delta(), **{name: _off(8)}) == INVALID
    assert _fwd(_delta(), beta=_off(1)) == INVALID
    assert _fwd(_delta(), ld=_off(2)) == INVALID
    assert _fwd(_delta(packed=1), cu=None) == INVALID
    assert _fwd(_delta(packed=1), cu=_off(2)) == INVALID
    for s in ((640 * 128, -128, 64), (640 * 128, 128, 32), (640 * 128, 132, 64)):
        pr = _delta()
        pr.sq[:] = s
        assert _fwd(pr) == INVALID
    for field in ("sbeta", "sdecay"):
        pr = _delta()
        getattr(pr, field)[1] = -1
        assert _fwd(pr) == INVALID
    pr = _delta()
    pr.so[2] = 0                                     # an output row twice
    assert _fwd(pr) == INVALID
    pr = _delta()
    need = K._lib().kata_fwd_delta_workspace_size(ctypes.byref(pr))
    assert need >= 2 * 4 * 10 * (1280 + 10240)       # 10 chunks of 2 sequences and 4 heads
    assert _fwd(pr, ws=False) == WORKSPACE
    assert _fwd(pr, ws_bytes=need - 1) == WORKSPACE
    a = _fake(9)
    assert _fwd(pr, sT=a[6]) == INVALID              # the final state over the initial one
    assert _fwd(pr, sT=ctypes.c_void_p(a[6].value + 64)) == INVALID
    # more workgroups than are numbered
    big = _delta(n_seq=65535, H=16500, Hk=16500, T=128, dk=8, dv=8, dtype=1)
    assert _fwd(big) == UNSUPPORTED


def test_delta_decode_and_backward_refusals():
    lib = K._lib()
    f = _fake(18)
    pr = _delta(T=1, packed=1)
    assert lib.kata_decode_delta(ctypes.byref(pr), *f[:7], None) == INVALID
    pr = _delta(T=1)
    for i in (0, 1, 2, 3, 5, 6):                     # q k v beta, state, o
        a = list(f[:7])
        a[i] = None
        assert lib.kata_decode_delta(ctypes.byref(pr), *a, None) == INVALID, i
    a = list(f[:7])
    a[5] = _off(4)
    assert lib.kata_decode_delta(ctypes.byref(pr), *a, None) == INVALID
    assert lib.kata_decode_delta(None, *f[:7], None) == INVALID
    pr = _delta()
    need = lib.kata_bwd_delta_workspace_size(ctypes.byref(pr))
    call = lambda a, n=need: lib.kata_bwd_delta(ctypes.byref(pr), *a, f[16], n, None)  # noqa: E731
    for i in (0, 1, 2, 3, 5, 9, 10, 11, 12):         # q k v beta dO, dq dk dv dbeta
        a = list(f[:15])
        a[i] = None
        assert call(a) == INVALID, i
    assert call(f[:15], need - 1) == WORKSPACE
    for read in (7, 8):                              # dinitial_state over the states that are read
        a = list(f[:15])
        a[14] = a[read]
        assert call(a) == INVALID
    assert lib.kata_bwd_delta(None, *f[:15], f[16], need, None) == INVALID


def _rot(B=2, T=3, H=2, Hk=1, D=16, rot=8, dtype=1):
    pr = KL._RotaryProblem()
    pr.B, pr.T, pr.H, pr.Hk, pr.D, pr.rot, pr.dtype, pr.magnitude = B, T, H, Hk, D, rot, dtype, 1.0
    pr.pos_b, pr.pos_t = T, 1
    pr.sq[:] = pr.soq[:] = (T * H * D, H * D, D)
    pr.sk[:] = pr.sok[:] = (T * Hk * D, Hk * D, D)
    return pr


def test_rotary_axes_refusals():
    lib, f = K._lib(), _fake(8)
    call = lambda q, k, rates, pos, axes, n, step, oq, ok: lib.kata_rotary_axes(  # noqa: E731
        ctypes.byref(_rot()), q, k, rates, pos, axes, n, step, oq, ok, None)
    good = [f[0], f[1], f[2], f[3], f[4], 3, 6, f[5], f[6]]
    for i, x in ((0, None), (1, None), (2, None), (3, None), (4, None), (4, _off(2)), (3, _off(2)), (5, 0), (6, -1), (7, None),
                 (8, None)):
        a = list(good)
        a[i] = x
        assert call(*a) == INVALID, i
    assert lib.kata_rotary_axes(None, *good, None) == INVALID


def _qkn(B=2, T=3, H=2, Hk=1, D=16, rot=8, dtype=1, w_dtype=0, eps=1e-6):
    pr = KD._QkNormProblem()
    for name, x in dict(B=B, T=T, H=H, Hk=Hk, D=D, rot=rot, dtype=dtype, w_dtype=w_dtype, eps=eps, magnitude=1.0, n_axes=1,
                        pos_b=T, pos_t=1).items():
        setattr(pr, name, x)
    pr.sq[:] = pr.soq[:] = pr.sdq[:] = (T * H * D, H * D, D)
    pr.sk[:] = pr.sok[:] = pr.sdk[:] = (T * Hk * D, Hk * D, D)
    return pr


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, INVALID), ("T", 0, INVALID), ("H", 0, INVALID), ("Hk", -1, INVALID), ("D", 0, INVALID), ("rot", 3, INVALID),
    ("rot", 18, INVALID), ("D", 258, UNSUPPORTED), ("H", 5000, UNSUPPORTED), ("dtype", 5, INVALID), ("w_dtype", 3, INVALID),
    ("magnitude", float("nan"), INVALID), ("eps", -1.0, INVALID), ("eps", float("inf"), INVALID), ("pos_t", -1, INVALID),
    ("pos_a", -1, INVALID),
])
def test_qk_norm_refuses_bad_problems(field, value, code):
    lib, pr = K._lib(), _qkn()
    setattr(pr, field, value)
    assert lib.kata_fwd_qk_norm(ctypes.byref(pr), *_fake(9), None) == code
    assert lib.kata_bwd_qk_norm_workspace_size(ctypes.byref(pr)) == 0


def test_qk_norm_refuses_bad_pointers_and_workspaces():
    lib, f = K._lib(), _fake(15)
    call = lambda a, pr=None: lib.kata_fwd_qk_norm(ctypes.byref(pr or _qkn()), *a, None)  # noqa: E731
    for i, x in ((0, None), (1, None), (4, None), (7, None), (8, None), (0, _off(1)), (2, _off(2)), (4, _off(4)), (5, _off(2)),
                 (6, _off(2))):                      # q k, rates, out q, out k; alignment of q, a weight, rates, positions, axes
        a = list(f[:9])
        a[i] = x
        assert call(a) == INVALID, (i, x)
    a = list(f[:9])
    a[5] = None                                      # axes without positions
    assert call(a) == INVALID
    assert lib.kata_fwd_qk_norm(None, *f[:9], None) == INVALID
    assert call(f[:9], _qkn(dtype=0, w_dtype=1)) == INVALID                # fp32 rows, bf16 weights
    pr = _qkn()
    pr.soq[1] = 0
    assert call(f[:9], pr) == INVALID
    pr = _qkn()
    need = lib.kata_bwd_qk_norm_workspace_size(ctypes.byref(pr))
    assert need == 768 * 2 * 16 * 4
    bwd = lambda a, n=need: lib.kata_bwd_qk_norm(ctypes.byref(pr), *a, n, None)  # noqa: E731
    for i in (0, 1, 2, 3, 6, 9, 10):                 # dq dk q k, rates, the gradients
        a = list(f[:14])
        a[i] = None
        assert bwd(a) == INVALID, i
    assert bwd(f[:14], need - 1) == WORKSPACE
    a = list(f[:14])
    a[13] = None
    assert bwd(a) == WORKSPACE
    pr.sdq[2] = 8
    assert bwd(f[:14]) == INVALID


def test_the_binding_refuses_cpu_tensors():
    q, b = torch.zeros(1, 4, 2, 16), torch.zeros(1, 4, 2)
    for bad in (lambda: K.fwd_delta(q, q, q, b), lambda: K.bwd_delta(q, q, q, b, q), lambda: K.fwd_qk_norm(q, q),
                lambda: K.decode_delta(q, q, q, b, torch.zeros(1, 2, 16, 16)), lambda: K.parallel_delta_attn(q, q, q, b),
                lambda: K.bwd_qk_norm(q, q, q, q), lambda: K.qk_norm_workspace_size(q)):
        with pytest.raises(ValueError):
            bad()


def test_rotary_axes_of_sections():
    assert K.rotary_axes((2, 1, 3), device="cpu").tolist() == [0, 0, 1, 2, 2, 2]
    assert K.rotary_axes((2, 1, 3), interleaved=True, device="cpu").tolist() == [0, 1, 2, 0, 2, 2]
    assert K.rotary_axes((0, 2), device="cpu").dtype == torch.int32
    for bad in ((), (1, -1)):
        with pytest.raises(ValueError):
            K.rotary_axes(bad, device="cpu")


@pytest.fixture(scope="module")
def fuzz_driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path_factory.mktemp("delta_fuzz") / "delta_fuzz")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "plan.cpp"),
           os.path.join(CSRC, "layer_plan.cpp"), os.path.join(CSRC, "delta_plan.cpp"),
           os.path.join(ROOT, "tests", "delta_fuzz.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("seed", [3, 77])
def test_the_planner_is_clean_under_sanitizers(fuzz_driver, seed):
    r = subprocess.run([fuzz_driver, str(seed), "200000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    _, n, _, valid, _, refused = r.stdout.split()
    assert int(valid) > 10000 and int(refused) > 10000
