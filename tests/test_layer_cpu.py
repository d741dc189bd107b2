"""The layer operators without a GPU: the C ABI's refusals (fake, never dereferenced pointers:
validation runs before any device call), the binding's refusals, and the planner under the host
sanitizers."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import kernelized_psd_feature_amd as K
from kernelized_psd_feature_amd import layer as KL

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kernelized_psd_feature_amd", "csrc")
OK, INVALID, UNSUPPORTED, WORKSPACE, DEVICE = 0, 1, 2, 3, 4
FAKE = 0x7F0000000000


def _fake(n):
    return [ctypes.c_void_p(FAKE + i * (1 << 32)) for i in range(n)]


def _decay(n_seq=2, H=2, T=640, dk=64, dv=64, packed=0, dtype=1, scale=1.0):
    pr = KL._DecayProblem()
    pr.n_seq, pr.H, pr.T, pr.dk, pr.dv, pr.packed, pr.dtype, pr.scale = n_seq, H, T, dk, dv, packed, dtype, scale
    for s, w in ((pr.sq, dk), (pr.sk, dk), (pr.sv, dv), (pr.so, dv), (pr.sdo, dv)):
        s[:] = (T * H * w, H * w, w)
    return pr


def _fwd(pr, ws=True, ws_bytes=None, **swap):
    lib = K._lib()
    q, k, v, ld, cu, s0, o, sT, w = _fake(9)
    a = dict(q=q, k=k, v=v, ld=ld, cu=cu, s0=s0, o=o, sT=sT)
    a.update(swap)
    need = lib.kata_fwd_decay_workspace_size(ctypes.byref(pr)) if pr is not None else 0
    return lib.kata_fwd_decay(ctypes.byref(pr) if pr is not None else None, *a.values(), w if ws else None,
                              need if ws_bytes is None else ws_bytes, None)


def _off(n):
    return ctypes.c_void_p(FAKE + n)


@pytest.mark.parametrize("field,value,code", [
    ("n_seq", 0, INVALID), ("H", 0, INVALID), ("T", 0, INVALID), ("dk", 0, INVALID), ("dv", -8, INVALID),
    ("dk", 12, UNSUPPORTED), ("dv", 136, UNSUPPORTED), ("T", (1 << 26) + 1, UNSUPPORTED),
    ("n_seq", 65536, UNSUPPORTED), ("dtype", 2, INVALID), ("packed", 2, INVALID),
    ("scale", float("nan"), INVALID), ("scale", float("inf"), INVALID),
])
def test_decay_refuses_bad_problems(field, value, code):
    pr = _decay()
    setattr(pr, field, value)
    assert _fwd(pr) == code
    assert K._lib().kata_last_error()


def test_decay_refuses_bad_pointers_strides_and_workspaces():
    assert _fwd(None) == INVALID
    for name in ("q", "k", "v", "ld", "o"):
        assert _fwd(_decay(), **{name: None}) == INVALID
    for name in ("q", "k", "v", "o", "s0", "sT"):
        assert _fwd(_decay(), **{name: _off(8)}) == INVALID
    assert _fwd(_decay(packed=1), cu=None) == INVALID
    assert _fwd(_decay(packed=1), cu=_off(2)) == INVALID
    for s, code in (((640 * 128, -128, 64), INVALID), ((640 * 128, 128, 32), INVALID), ((640 * 128, 132, 64), INVALID)):
        pr = _decay()
        pr.sq[:] = s
        assert _fwd(pr) == code
    pr = _decay()
    pr.so[2] = 0                                     # an output row twice
    assert _fwd(pr) == INVALID
    pr = _decay()
    need = K._lib().kata_fwd_decay_workspace_size(ctypes.byref(pr))
    assert need > 0                                  # 10 chunks, 4 sequences x heads: segments
    assert _fwd(pr, ws=False) == WORKSPACE
    assert _fwd(pr, ws_bytes=need - 1) == WORKSPACE
    pr.T = 64
    assert K._lib().kata_fwd_decay_workspace_size(ctypes.byref(pr)) == 0


def test_decay_accepts_broadcast_inputs():
    pr = _decay()
    pr.sk[2] = 0                                     # all heads share their keys
    pr.sv[0] = 0
    assert _fwd(pr) == DEVICE or torch.cuda.is_available()


def test_decode_and_backward_refusals():
    lib = K._lib()
    f = _fake(14)
    pr = _decay(T=1, packed=1)
    assert lib.kata_decode_decay(ctypes.byref(pr), f[0], f[1], f[2], f[3], f[4], f[5], None) == INVALID
    pr = _decay(T=1)
    assert lib.kata_decode_decay(ctypes.byref(pr), f[0], f[1], f[2], f[3], None, f[5], None) == INVALID
    assert lib.kata_decode_decay(ctypes.byref(pr), f[0], f[1], f[2], f[3], _off(4), f[5], None) == INVALID
    pr = _decay()
    need = lib.kata_bwd_decay_workspace_size(ctypes.byref(pr))
    call = lambda a, n=need: lib.kata_bwd_decay(ctypes.byref(pr), *a, f[13], n, None)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 8, 9, 10):              # q k v dO log_decay, dq dk dv
        a = list(f[:12])
        a[i] = None
        assert call(a) == INVALID, i
    assert call(f[:12], need - 1) == WORKSPACE


@pytest.mark.parametrize("n_seq,H,dtype,d", [
    (65535, 65535, 1, 8), (65535, 40000, 1, 8), (65535, 20000, 0, 128),   # two blocks of columns
])
def test_decay_refuses_more_workgroups_than_it_can_number(n_seq, H, dtype, d):
    pr = _decay(n_seq=n_seq, H=H, T=1, dk=d, dv=d, dtype=dtype)
    assert _fwd(pr) == UNSUPPORTED
    assert b"one launch" in K._lib().kata_last_error()


def test_decay_refuses_states_that_overlap():
    size = 2 * 2 * 64 * 64 * 4
    s0 = _fake(9)[5].value
    for by in (-size + 16, -16, 16, size - 16):      # the same array at another place
        assert _fwd(_decay(), sT=ctypes.c_void_p(s0 + by)) == INVALID
        assert b"overlaps" in K._lib().kata_last_error()
    if not torch.cuda.is_available():                # (made-up addresses: nothing may be launched on them)
        for by in (-size, 0, size):
            assert _fwd(_decay(), sT=ctypes.c_void_p(s0 + by)) == DEVICE
    lib, f, pr = K._lib(), _fake(14), _decay()
    need = lib.kata_bwd_decay_workspace_size(ctypes.byref(pr))
    for i in (6, 7):                                 # initial_state, dfinal_state
        for by in (-16, 0, size - 16):
            a = list(f[:12])
            a[11] = ctypes.c_void_p(f[i].value + by)
            assert lib.kata_bwd_decay(ctypes.byref(pr), *a, f[13], need, None) == INVALID
            assert b"overlaps" in lib.kata_last_error()


def test_decode_takes_any_number_of_sequences():
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real: nothing may be launched on them")
    f, pr = _fake(6), _decay(n_seq=1 << 20, H=1, T=1, dk=16, dv=16)
    assert K._lib().kata_decode_decay(ctypes.byref(pr), *f, None) == DEVICE
    pr.H = 65536
    assert K._lib().kata_decode_decay(ctypes.byref(pr), *f, None) == UNSUPPORTED


def _rot(B=2, T=3, H=4, Hk=2, D=16, rot=16, dtype=1):
    pr = KL._RotaryProblem()
    pr.B, pr.T, pr.H, pr.Hk, pr.D, pr.rot, pr.dtype, pr.magnitude = B, T, H, Hk, D, rot, dtype, 1.0
    pr.sq[:] = pr.soq[:] = (T * H * D, H * D, D)
    pr.sk[:] = pr.sok[:] = (T * Hk * D, Hk * D, D)
    return pr


@pytest.mark.parametrize("field,value,code", [
    ("B", 0, INVALID), ("T", 0, INVALID), ("H", 0, INVALID), ("Hk", -1, INVALID), ("D", 0, INVALID),
    ("rot", 3, INVALID), ("rot", 18, INVALID), ("rot", -2, INVALID), ("D", 1026, UNSUPPORTED),
    ("H", 5000, UNSUPPORTED), ("dtype", 5, INVALID), ("magnitude", float("nan"), INVALID),
    ("pos_t", -1, INVALID),
])
def test_rotary_refuses_bad_problems(field, value, code):
    pr = _rot()
    setattr(pr, field, value)
    assert K._lib().kata_rotary(ctypes.byref(pr), *_fake(6), None) == code


def test_rotary_refuses_bad_pointers():
    lib, f = K._lib(), _fake(6)
    for i in (0, 1, 2, 4, 5):                        # q k rates, out q, out k
        a = list(f)
        a[i] = None
        assert lib.kata_rotary(ctypes.byref(_rot()), *a, None) == INVALID, i
    for i in (0, 1, 2, 3, 4, 5):
        a = list(f)
        a[i] = _off(1)
        assert lib.kata_rotary(ctypes.byref(_rot()), *a, None) == INVALID, i
    pr = _rot()
    pr.soq[1] = 0
    assert lib.kata_rotary(ctypes.byref(pr), *f, None) == INVALID
    assert lib.kata_rotary(None, *f, None) == INVALID


def _norm(rows=5, N=64, dtype=1, w_dtype=0, eps=1e-5):
    pr = KL._NormProblem()
    pr.rows, pr.N, pr.dtype, pr.w_dtype, pr.eps = rows, N, dtype, w_dtype, eps
    pr.sx = pr.sy = pr.sdy = pr.sdx = N
    return pr


@pytest.mark.parametrize("field,value,code", [
    ("rows", 0, INVALID), ("N", 0, INVALID), ("N", 1 << 25, UNSUPPORTED), ("dtype", 3, INVALID),
    ("w_dtype", 3, INVALID), ("eps", -1.0, INVALID), ("eps", float("nan"), INVALID), ("sx", -64, INVALID),
    ("sy", 0, INVALID), ("sx", 32, INVALID),
])
def test_norm_refuses_bad_problems(field, value, code):
    lib, pr = K._lib(), _norm()
    setattr(pr, field, value)
    assert lib.kata_fwd_layer_norm(ctypes.byref(pr), *_fake(6), None) == code
    assert lib.kata_bwd_layer_norm_workspace_size(ctypes.byref(pr)) == 0


def test_norm_refuses_bad_pointers():
    lib, f = K._lib(), _fake(9)
    pr = _norm()
    call = lambda a: lib.kata_fwd_layer_norm(ctypes.byref(pr), *a, None)  # noqa: E731
    for i in (0, 3, 4):                              # x, y, mean without rstd
        a = list(f[:6])
        a[i] = None
        assert call(a) == INVALID, i
    need = lib.kata_bwd_layer_norm_workspace_size(ctypes.byref(pr))
    bwd = lambda a, n=need: lib.kata_bwd_layer_norm(ctypes.byref(pr), *a, n, None)  # noqa: E731
    for i in (0, 1, 3, 4):
        a = list(f)
        a[i] = None
        assert bwd(a) == INVALID, i
    a = list(f)
    a[5] = a[6] = a[7] = None
    assert bwd(a) == INVALID
    assert bwd(f, need - 1) == WORKSPACE
    assert lib.kata_bwd_layer_norm(ctypes.byref(pr), *f[:8], None, need, None) == WORKSPACE
    pr = _norm(dtype=0, w_dtype=1)                   # fp32 rows, bf16 weights
    assert call(f[:6]) == INVALID


@pytest.mark.parametrize("rows", [1, 63, 64, 65, 1 << 20])
@pytest.mark.parametrize("N,most", [(1024, 768), (8192, 768), (8193, 64), (1 << 20, 64)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_norm_workspace_holds_the_partial_rows_that_there_are(dtype, N, most, rows):
    # a pair of fp32 rows a workgroup, in whole 256 bytes: of wide rows there are 64 workgroups
    pr = _norm(rows=rows, N=N, dtype=dtype)
    need = min(rows, most) * 2 * N * 4
    got = K._lib().kata_bwd_layer_norm_workspace_size(ctypes.byref(pr))
    assert need <= got < need + 256


def test_the_binding_refuses_cpu_tensors_and_bad_rates():
    q = torch.zeros(1, 4, 2, 16)
    with pytest.raises(ValueError):
        K.fwd_decay(q, q, q, torch.zeros(2))
    with pytest.raises(ValueError):
        K.rotary(q, q, torch.zeros(8, dtype=torch.float64))
    with pytest.raises(ValueError):
        K.fwd_layer_norm(q)
    for kw in (dict(dim=3), dict(dim=0), dict(dim=2, scaling="ntk", factor=2.0), dict(dim=8, scaling="cube"),
               dict(dim=8, factor=0.5), dict(dim=8, scaling="parts"), dict(dim=8, base=0.0),
               dict(dim=8, scaling="parts", original_length=64, low=3.0, high=3.0)):
        with pytest.raises(ValueError):
            K.rotary_rates(device="cpu", **kw)


def test_rotary_rates_scalings():
    plain, m = K.rotary_rates(16, device="cpu")
    assert m == 1.0 and plain[0] == 1.0 and plain.dtype == torch.float64
    lin, _ = K.rotary_rates(16, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(lin, plain / 4)
    ntk, _ = K.rotary_rates(16, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and abs(float(ntk[-1] / plain[-1]) - 0.25) < 1e-12
    parts, m = K.rotary_rates(16, scaling="parts", factor=4.0, original_length=4096, device="cpu")
    assert parts[0] == plain[0] and parts[-1] == plain[-1] / 4 and m > 1.0
    assert torch.all(parts <= plain) and torch.all(parts >= plain / 4)


@pytest.fixture(scope="module")
def fuzz_driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path_factory.mktemp("layer_fuzz") / "layer_fuzz")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "plan.cpp"),
           os.path.join(CSRC, "layer_plan.cpp"), os.path.join(ROOT, "tests", "layer_fuzz.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("seed", [3, 77])
def test_the_planner_is_clean_under_sanitizers(fuzz_driver, seed):
    r = subprocess.run([fuzz_driver, str(seed), "200000"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    _, n, _, valid, _, refused = r.stdout.split()
    assert int(valid) > 10000 and int(refused) > 10000
