"""What the layers take as their rotary argument, and rotations without a pair."""

import pytest
import torch

import kernelized_psd_feature_amd as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def _layers(q, v, b, rotary, positions):
    decay = torch.full((q.shape[2],), -0.1, device=DEV)
    return (lambda: K.parallel_kata_attn(q, q, v, rotary=rotary, positions=positions),
            lambda: K.parallel_decay_attn(q, q, v, decay, rotary=rotary, positions=positions),
            lambda: K.parallel_delta_attn(q, q, v, b, rotary=rotary, positions=positions),
            lambda: K.parallel_delta_attn(q, q, v, b, rotary=rotary, positions=positions, qk_norm="l2"))


def test_tables_of_another_length_are_refused():
    q = torch.full((1, 64, 2, 16), 0.25, device=DEV)    # keys of unit length
    b, (rates, magnitude) = torch.ones(1, 64, 2, device=DEV), K.rotary_rates(16)
    axes, pos = K.rotary_axes((4, 4)), torch.zeros(2, 1, 64, dtype=torch.int32, device=DEV)
    for table in ((rates,), (rates, magnitude, axes, 0), (), rates, {"rates": rates, "magnitude": 1.0}):
        for call in _layers(q, q, b, table, pos):
            with pytest.raises(ValueError):
                call()
    for call in (*_layers(q, q, b, (rates, magnitude, axes), pos), *_layers(q, q, b, [rates, magnitude], pos[0]),
                 *_layers(q, q, b, (rates, magnitude, None), pos[0])):
        assert torch.isfinite(call()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_pair_of_several_axes_is_a_copy(dtype):
    q = torch.randn(2, 5, 3, 16, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    rates, axes = torch.empty(0, dtype=torch.float64, device=DEV), K.rotary_axes((0, 0))
    pos = torch.ones(2, 2, 5, dtype=torch.int64, device=DEV)
    a, b = K.rotary(q, q[:, :, :1], rates, positions=pos, axes=axes)
    assert torch.equal(a, q) and torch.equal(b, q[:, :, :1])
    assert torch.equal(K.fwd_qk_norm(q, None, rates=rates, positions=pos, axes=axes), K.fwd_qk_norm(q, None))
