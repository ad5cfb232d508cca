"""The torch layer of layer norm and its checkpoint on the GPU: what a call
refuses, what a refused call leaves alone, and what it raises."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def norm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gradients_taco_compress_amd.norm as norm
    return norm


def announce(msg):
    print(f"[case] {msg}", flush=True)


def randn(*shape, dtype=BF, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


@pytest.mark.parametrize("other_stream", [False, True])
def test_a_tensor_of_the_right_size_and_the_wrong_shape_is_refused(norm, other_stream):
    """[hidden, out_features] is no gradient buffer of [out_features, hidden],
    [hidden, rows] no checkpoint of [rows, hidden]; both paths to the C ABI."""
    announce(f"wrong shapes, {'general' if other_stream else 'usual'} path")
    stream = torch.cuda.current_stream() if other_stream else None
    x, dz = randn(6, 64), randn(6, 24, seed=1)
    y, codes, rstd = norm.layer_norm_checkpoint(x)
    turned = torch.full((64, 24), 7.0, device="cuda")
    for accumulate in (False, True):
        with pytest.raises(ValueError, match="out must be"):
            norm.checkpoint_weight_grad(dz, codes, out=turned, dtype=F32, accumulate=accumulate,
                                        stream=stream)
    assert bool(turned.eq(7.0).all())
    with pytest.raises(ValueError, match="codes must hold rows"):
        norm.layer_norm_checkpoint_backward(y, codes.reshape(64, 6), rstd, stream=stream)
    with pytest.raises(ValueError, match="codes must hold rows"):
        norm.layer_norm_checkpoint(x, codes=codes.reshape(64, 6), stream=stream)
    # Rows may be spread over any leading dimensions.
    kept = norm.layer_norm_checkpoint(x.view(2, 3, 64), codes=codes, stream=stream)
    assert kept[1] is codes
    dx, _, _ = norm.layer_norm_checkpoint_backward(y.view(3, 2, 64), codes, rstd, stream=stream)
    assert dx.shape == (3, 2, 64)
    out = torch.zeros(24, 64, device="cuda")
    got, _ = norm.checkpoint_weight_grad(dz.view(2, 3, 24), codes, out=out, stream=stream)
    assert got is out and torch.equal(out, norm.checkpoint_weight_grad(dz, codes, dtype=F32)[0])


@pytest.mark.parametrize("dy_type,wanted", [(BF, F16), (F16, BF)])
def test_a_refused_type_leaves_out_alone(norm, dy_type, wanted):
    """dtype names a type that dW cannot have: nothing is written or launched."""
    announce(f"refused type {wanted}")
    _, codes, _ = norm.layer_norm_checkpoint(randn(6, 64))
    dz = randn(6, 24, dtype=dy_type)
    out = torch.full((24, 64), 7.0, device="cuda", dtype=dy_type)
    with pytest.raises(TypeError, match="dtype must be"):
        norm.checkpoint_weight_grad(dz, codes, out=out, dtype=wanted)
    assert bool(out.eq(7.0).all())
    with pytest.raises(TypeError, match="dtype must be"):
        norm.checkpoint_weight_grad(dz, codes, dtype=wanted)
    # out of another type than the one named.
    with pytest.raises(TypeError, match="out must be"):
        norm.checkpoint_weight_grad(dz, codes, out=out, dtype=F32)
    assert bool(out.eq(7.0).all())


def test_running_out_of_memory_has_its_own_type(norm):
    """Callers catch torch.OutOfMemoryError: half a tebibyte of dW is not there."""
    announce("out of memory")
    n = 1 << 19
    dz = torch.zeros(1, n, device="cuda", dtype=BF)
    codes = torch.zeros(1, n, device="cuda", dtype=torch.uint8)
    with pytest.raises(torch.OutOfMemoryError):
        norm.checkpoint_weight_grad(dz, codes)
