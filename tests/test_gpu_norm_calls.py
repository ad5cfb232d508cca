"""The torch layer of layer norm and its checkpoint on the GPU: what a call
refuses, what a refused call leaves alone, and what it raises."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

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


STUB = r"""
#include <stdint.h>
int stub_calls = 0;
#define FAILS(name) int name(void) { ++stub_calls; return 7; }
FAILS(taco_norm_forward) FAILS(taco_norm_checkpoint) FAILS(taco_norm_backward)
FAILS(taco_norm_checkpoint_backward) FAILS(taco_norm_weight_grad)
float taco_norm_checkpoint_scale(int64_t hidden) { (void)hidden; return 1.0f; }
int64_t taco_norm_backward_workspace(int64_t rows, int64_t hidden) { return 16 + 0 * rows * hidden; }
int64_t taco_norm_weight_grad_workspace(void) { return 16; }
"""

CHILD = r"""
import ctypes
import torch
from gradients_taco_compress_amd import norm
calls = ctypes.c_int.in_dll(norm._lib, "stub_calls")
x = torch.ones(4, 64, device="cuda", dtype=torch.bfloat16)
one = torch.ones(4, device="cuda")
codes = torch.zeros(4, 64, device="cuda", dtype=torch.uint8)
acc = torch.zeros(64, 64, device="cuda")
for name, call in (("taco_norm_forward", lambda: norm.layer_norm(x)),
                   ("taco_norm_checkpoint", lambda: norm.layer_norm_checkpoint(x)),
                   ("taco_norm_backward", lambda: norm.layer_norm_backward(x, x, one, one)),
                   ("taco_norm_checkpoint_backward",
                    lambda: norm.layer_norm_checkpoint_backward(x, codes, one)),
                   ("taco_norm_weight_grad", lambda: norm.checkpoint_weight_grad(
                       x, codes, out=acc, accumulate=True))):
    calls.value = 0
    try:
        call()
        print(name, "returned", flush=True)
    except norm.TacoError as e:
        print(name, e.status, calls.value, name in str(e), flush=True)
"""


def test_a_failed_launch_is_reported_and_not_made_again(norm, tmp_path):
    """A launch that fails may follow one that did not (a gradient that is
    already added to): the call is over.  The library is a stub here whose calls
    all report TACO_ERR_HIP and launch nothing."""
    announce("failed launch")
    package = tmp_path / "gradients_taco_compress_amd"
    package.mkdir()
    for f in os.listdir(norm.PKG):
        if f.endswith((".py", ".so")) and f != "libtaco_norm.so":
            shutil.copy(os.path.join(norm.PKG, f), package / f)
    (tmp_path / "stub.c").write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-w", "-Wl,-soname,libtaco_norm.so",
                    str(tmp_path / "stub.c"), "-o", str(package / "libtaco_norm.so")], check=True)
    out = subprocess.run([sys.executable, "-c", CHILD], cwd=tmp_path, capture_output=True, text=True,
                         timeout=110, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert out.returncode == 0, out.stderr
    names = ("forward", "checkpoint", "backward", "checkpoint_backward", "weight_grad")
    assert out.stdout.split("\n")[:-1] == [f"taco_norm_{n} 7 1 True" for n in names]


# ---------------------------------------------------- slices of one buffer --

def test_interleaved_column_slices_are_apart(norm):
    """Inputs and outputs side by side in one buffer, no element shared."""
    announce("column slices of one buffer")
    rows, hidden = 300, 136
    buf = randn(rows, 4 * hidden)
    x, y, dy, dx = (buf[:, i * hidden:(i + 1) * hidden] for i in range(4))
    dy0 = dy.clone()
    want = norm.layer_norm(x.contiguous())
    got = norm.layer_norm(x, out=y)
    assert got[0] is y and all(torch.equal(a, b) for a, b in zip(got, want))
    _, mean, rstd = want
    want = norm.layer_norm_backward(dy0, x.contiguous(), mean, rstd)
    got = norm.layer_norm_backward(dy, x, mean, rstd, dx=dx)
    assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(dy, dy0)
    for out in (buf[:, hidden // 2:hidden // 2 + hidden], buf[:, 1:1 + hidden], x):
        with pytest.raises(norm.TacoError, match="ALIAS"):
            norm.layer_norm(x, out=out)


# --------------------------------------------------------------- autograd --

def test_gradients_have_their_parameter_s_shape(norm):
    announce("parameter shapes")
    x, W, c = randn(6, 64), randn(24, 64, seed=1).requires_grad_(), randn(24, seed=2)
    w = randn(64, dtype=F32, seed=3)
    for shape in ((64,), (1, 64), (64, 1)):
        weight, bias = w.view(shape).clone().requires_grad_(), w.view(shape).clone().requires_grad_()
        for out in (norm.norm(x, weight, bias), norm.norm_linear(x, weight, bias, W)):
            grads = torch.autograd.grad(out.float().square().sum(), (weight, bias))
            assert all(g.shape == shape for g in grads)
    with pytest.raises(ValueError, match="linear_weight"):
        norm.norm_linear(x, None, None, W[0])
    with pytest.raises(ValueError, match="linear_weight"):
        norm.norm_linear(x, None, None, W[:, :32])
    for bias in (c[:1], c.view(1, 24)):
        with pytest.raises(ValueError, match="linear_bias"):
            norm.norm_linear(x, None, None, W, bias)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.mark.parametrize("inside", [False, True])
@pytest.mark.parametrize("dtype,ptype,leaf,auto", [(BF, F32, BF, F16), (BF, BF, F32, F16),
                                                   (F16, F16, F32, BF), (BF, F32, F32, BF),
                                                   (F32, F32, F32, BF), (F32, F32, F32, F16)])
def test_norm_linear_under_autocast(norm, dtype, ptype, leaf, auto, inside):
    """As torch's own layers there: the norm in its input's type, the linear
    layer in autocast's, gradients in the leaves' types.  Backward inside and
    outside of the region.

    Against the formulas in 64 bits with the checkpoint's h and the linear
    weight as cast.  A result is rounded to autocast's type, to the activation's
    (dy) and to its leaf's: half a step each, in the 2-norm."""
    announce(f"autocast {dtype} {leaf} under {auto}, backward {'inside' if inside else 'outside'}")
    rows, hidden, features = 96, 160, 72
    x = (randn(4, 24, hidden, dtype=F32, seed=5) * 1.5 + 0.3).to(dtype).requires_grad_()
    w = (1 + 0.3 * randn(hidden, dtype=F32, seed=6)).to(ptype).requires_grad_()
    b = randn(hidden, dtype=ptype, seed=7).requires_grad_()
    W = (0.05 * randn(features, hidden, dtype=F32, seed=8)).to(leaf).requires_grad_()
    c = randn(features, dtype=leaf, seed=9).requires_grad_()
    dz = randn(4, 24, features, dtype=auto, seed=10)
    with torch.autocast("cuda", dtype=auto):
        z = norm.norm_linear(x, w, b, W, c)
        assert z.dtype == auto and z.shape == dz.shape
        if inside:
            got = torch.autograd.grad(z, (x, w, b, W, c), dz)
    if not inside:
        got = torch.autograd.grad(z, (x, w, b, W, c), dz)
    with torch.no_grad():
        y, codes, rstd = norm.layer_norm_checkpoint(x, w, b)
        assert torch.equal(z, torch.nn.functional.linear(y.to(auto), W.to(auto), c.to(auto)))
        h = codes.view(torch.float8_e4m3fn).double().view(rows, hidden) / norm.checkpoint_scale(hidden)
        d, r64 = dz.double().view(rows, features), rstd.double()[:, None]
        g = (d @ W.to(auto).double()) * w.double()
        dx = r64 * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        dy = d @ W.to(auto).double()
        want = (dx.view(x.shape), (dy * h).sum(0), dy.sum(0),
                d.t() @ (h * w.double() + b.double()), d.sum(0))
    for name, leaf_t, a, r in zip("xwbWc", (x, w, b, W, c), got, want):
        assert a.dtype == leaf_t.dtype and a.shape == leaf_t.shape
        bound = half_step(auto) + half_step(dtype) + half_step(leaf_t.dtype)
        assert float((a.double() - r).norm() / r.norm()) <= bound, name


def test_norm_linear_without_autocast_wants_one_type(norm):
    announce("types without autocast")
    x, W = randn(6, 64), randn(24, 64, dtype=F32)
    with pytest.raises(TypeError, match="linear_weight must be"):
        norm.norm_linear(x, None, None, W)
    with pytest.raises(TypeError, match="x must be"):
        norm.norm_linear(x.float(), None, None, W)
    with torch.autocast("cuda", enabled=False), pytest.raises(TypeError, match="linear_weight must be"):
        norm.norm_linear(x, None, None, W)
