"""libtaco_norm without a GPU: its C ABI refuses every bad argument before
touching the device, and the torch layer refuses what it cannot pass on."""
import ctypes
import os
import re
import subprocess
from fractions import Fraction

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
if torch.cuda.device_count() > 0:
    # Fake device pointers below: only where no kernel could run on them.
    pytest.skip("host-only validation tests (fake device pointers)", allow_module_level=True)
norm = pytest.importorskip("gradients_taco_compress_amd.norm")

HEADER = os.path.join(ROOT, "include", "taco_norm.h")
OK, NULL, SHAPE, BLOCK, PARAM, ALIGN, ALIAS, HIP, FORMAT = range(9)
BF16, F16, F32 = range(3)
A = 1 << 24          # spacing of fake, aligned device addresses


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(taco_norm_[a-z0-9_]+)\s*\(", text)))


def test_every_declared_function_is_exported_and_bound():
    out = subprocess.run(["nm", "-D", "--defined-only", norm.LIB_PATH], capture_output=True,
                         text=True).stdout
    assert set(re.findall(r" T (taco_\w+)", out)) == set(declared()) == set(norm.EXPORTS)
    for n in declared():
        assert callable(getattr(norm, n))


def test_norm_sources_compile_like_the_rest(monkeypatch, tmp_path):
    import __graft_entry__ as g
    m = g._load_hip_build()
    cmds = []

    def fake_run(cmd, verbose):
        cmds.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
    monkeypatch.setattr(m, "_run", fake_run)
    monkeypatch.setattr(m, "NORM_LIB", str(tmp_path / "libtaco_norm.so"))
    monkeypatch.setattr(m, "NORM_TORCH", str(tmp_path / "_norm_torch.so"))
    m.build_norm()
    compiles = [c for c in cmds if "-c" in c]
    assert sorted(c[c.index("-c") + 1] for c in compiles) == sorted(m.NORM_SOURCES)
    feature = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    for c in compiles:
        assert "--offload-arch=gfx950" in c and "-O3" in c
        assert any(c[i:i + 4] == feature for i in range(len(c) - 3))
    assert not [f for f in os.listdir(m.CSRC) if ".tmp" in f]


@pytest.mark.parametrize("hidden", [1, 2, 12, 13, 195, 196, 197, 784, 785, 2560, 12288, 12544,
                                    12545, 200704, 200705, 802816, 802817, 1048576])
def test_scale_is_the_largest_power_that_cannot_overflow(hidden):
    s = Fraction(norm.checkpoint_scale(hidden))
    assert hidden * s * s <= 448 * 448 < hidden * 4 * s * s


def test_scale_of_a_bad_width():
    for h in (0, -1, 1048577):
        assert norm.taco_norm_checkpoint_scale(h) == 0.0
        with pytest.raises(norm.TacoError, match="SHAPE"):
            norm.checkpoint_scale(h)


def forward(x=A, ldx=64, rows=4, hidden=64, dtype=BF16, w=2 * A, b=3 * A, pdtype=F32, eps=1e-5,
            y=4 * A, ldy=64, mean=5 * A, rstd=6 * A):
    return norm.taco_norm_forward(x, ldx, rows, hidden, dtype, w, b, pdtype, eps, y, ldy, mean,
                                  rstd, 0)


def checkpoint(x=A, ldx=64, rows=4, hidden=64, dtype=BF16, w=2 * A, b=3 * A, pdtype=F32, eps=1e-5,
               y=4 * A, ldy=64, codes=5 * A, rstd=6 * A):
    return norm.taco_norm_checkpoint(x, ldx, rows, hidden, dtype, w, b, pdtype, eps, y, ldy, codes,
                                     rstd, 0)


@pytest.mark.parametrize("call", [forward, checkpoint])
def test_forward_refusals(call):
    assert call(dtype=3) == FORMAT and call(dtype=-1) == FORMAT
    assert call(pdtype=F16) == FORMAT                      # bf16 with fp16 parameters
    assert call(dtype=F32, pdtype=BF16) == FORMAT
    assert call(hidden=0, ldx=0) == SHAPE and call(hidden=1048577) == SHAPE
    assert call(rows=-1) == SHAPE
    assert call(ldx=63) == SHAPE and call(ldy=63) == SHAPE
    assert call(ldx=1 << 50) == SHAPE
    for eps in (-1e-9, float("nan"), float("inf")):
        assert call(eps=eps) == PARAM
    assert call(x=0) == NULL and call(y=0) == NULL
    assert call(x=A + 1) == ALIGN and call(y=4 * A + 1) == ALIGN
    assert call(w=2 * A + 2) == ALIGN and call(b=3 * A + 1) == ALIGN
    assert call(rstd=6 * A + 2) == ALIGN
    assert call(y=A + 64) == ALIAS                          # y over x
    assert call(rstd=4 * A + 16) == ALIAS                   # rstd over y
    assert call(w=4 * A) == ALIAS
    assert call(rows=0, x=0, y=0) == OK


def test_checkpoint_needs_its_outputs():
    assert checkpoint(codes=0) == NULL and checkpoint(rstd=0) == NULL
    assert checkpoint(codes=4 * A + 100) == ALIAS
    assert checkpoint(codes=6 * A - 4 * 64 + 1) == ALIAS    # reaches into rstd


def backward(dy=A, lddy=64, x=2 * A, ldx=64, mean=3 * A, rstd=4 * A, w=5 * A, rows=4, hidden=64,
             dtype=BF16, pdtype=F32, dx=6 * A, lddx=64, dw=7 * A, db=8 * A, ws=9 * A, nbytes=None):
    nbytes = norm.taco_norm_backward_workspace(rows, hidden) if nbytes is None else nbytes
    return norm.taco_norm_backward(dy, lddy, x, ldx, mean, rstd, w, rows, hidden, dtype, pdtype,
                                   dx, lddx, dw, db, ws, nbytes, 0)


def backward_codes(dy=A, lddy=64, x=2 * A, rstd=4 * A, w=5 * A, rows=4, hidden=64, dtype=BF16,
                   pdtype=F32, dx=6 * A, lddx=64, dw=7 * A, db=8 * A, ws=9 * A, nbytes=None):
    nbytes = norm.taco_norm_backward_workspace(rows, hidden) if nbytes is None else nbytes
    return norm.taco_norm_checkpoint_backward(dy, lddy, x, rstd, w, rows, hidden, dtype, pdtype,
                                              dx, lddx, dw, db, ws, nbytes, 0)


@pytest.mark.parametrize("call", [backward, backward_codes])
def test_backward_refusals(call):
    assert call(dtype=7) == FORMAT and call(pdtype=F16) == FORMAT
    assert call(rows=-1, nbytes=0) == SHAPE and call(lddy=63) == SHAPE and call(lddx=1) == SHAPE
    for name in ("dy", "x", "rstd", "dx", "ws"):
        assert call(**{name: 0}) == NULL, name
    assert call(dy=A + 1) == ALIGN and call(ws=9 * A + 8) == ALIGN
    assert call(dw=7 * A + 2) == ALIGN and call(rstd=4 * A + 1) == ALIGN
    assert call(dx=A + 2) == ALIAS                          # shifted over dy
    assert call(dx=A, lddx=72) == ALIAS                     # dy's place, another pitch
    assert call(dx=2 * A) == ALIAS                          # over the saved activation
    assert call(dw=8 * A + 4) == ALIAS and call(ws=A) == ALIAS
    need = norm.taco_norm_backward_workspace(4, 64)
    assert need > 0 and call(nbytes=need - 1) == PARAM


def test_backward_of_the_input_alone_needs_x_and_mean():
    assert backward(mean=0) == NULL and backward(ldx=60) == SHAPE
    assert backward(mean=3 * A + 2) == ALIGN


def test_backward_workspace():
    f = norm.taco_norm_backward_workspace
    assert f(0, 64) == 0
    assert f(-1, 64) == f(4, 0) == f(4, 1048577) == f(1 << 47, 1 << 10) == -1
    assert f(1, 2560) == 2 * 2560 * 4
    assert f(1 << 20, 2560) == 512 * 2 * 2560 * 4


def weight_grad(dy=A, lddy=64, codes=2 * A, rows=4096, features=64, hidden=64, dtype=BF16, w=3 * A,
                b=4 * A, pdtype=F32, dw=5 * A, dwtype=BF16, accumulate=0, db=6 * A, ws=7 * A,
                nbytes=None):
    if nbytes is None:
        nbytes = norm.taco_norm_weight_grad_workspace(dy, lddy, codes, rows, features, hidden)
    return norm.taco_norm_weight_grad(dy, lddy, codes, rows, features, hidden, dtype, w, b, pdtype,
                                      dw, dwtype, accumulate, db, ws, nbytes, 0)


def test_weight_grad_refusals():
    assert weight_grad(dtype=F32, dwtype=F32) == FORMAT     # no matrix instruction for it
    assert weight_grad(dwtype=F16) == FORMAT and weight_grad(dwtype=5) == FORMAT
    assert weight_grad(accumulate=1) == FORMAT              # into bf16
    assert weight_grad(pdtype=F16) == FORMAT
    assert weight_grad(features=0, lddy=0) == SHAPE and weight_grad(hidden=0) == SHAPE
    assert weight_grad(lddy=63) == SHAPE and weight_grad(rows=-2, nbytes=0) == SHAPE
    for name in ("dy", "codes", "dw", "ws"):
        assert weight_grad(**{name: 0}) == NULL, name
    assert weight_grad(dy=A + 1) == ALIGN and weight_grad(dw=5 * A + 1) == ALIGN
    assert weight_grad(ws=7 * A + 4) == ALIGN and weight_grad(db=6 * A + 2) == ALIGN
    assert weight_grad(dw=A + 64) == ALIAS and weight_grad(db=5 * A) == ALIAS
    assert weight_grad(ws=2 * A) == ALIAS
    f = norm.taco_norm_weight_grad_workspace
    need = f(A, 64, 2 * A, 4096, 64, 64)                           # one tile, split
    assert need > 0 and weight_grad(nbytes=need - 1) == PARAM
    assert weight_grad(rows=4, nbytes=-1) == PARAM                 # needs none
    assert f(A, 64, 2 * A, 0, 64, 64) == 0 and f(A, 64, 2 * A, 4, 64, 64) == 0
    assert f(A, 0, 2 * A, 4, 0, 64) == f(A, 64, 2 * A, 4, 64, 0) == -1
    assert f(A, 64, 2 * A, -1, 64, 64) == f(A, 63, 2 * A, 4, 64, 64) == -1


def test_weight_grad_copies_operands_that_are_not_aligned():
    f = norm.taco_norm_weight_grad_workspace
    assert f(A + 2, 64, 2 * A, 4, 64, 64) == 4 * 128               # dy off by an element
    assert f(A, 65, 2 * A, 4, 64, 64) == 4 * 128                   # its rows
    assert f(A, 80, 2 * A, 4, 63, 64) == 4 * 128                   # its width
    assert f(A, 64, 2 * A + 1, 4, 64, 64) == 4 * 64                # codes
    assert f(A, 64, 2 * A, 4, 64, 40) == 4 * 48
    assert f(A, 65, 2 * A, 4, 65, 65) == 4 * (144 + 80)


def test_torch_layer_refuses_host_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: norm.layer_norm(x), lambda: norm.layer_norm_checkpoint(x),
                 lambda: norm.layer_norm_backward(x, x, x[:, 0], x[:, 0]),
                 lambda: norm.layer_norm_checkpoint_backward(x, x, x[:, 0]),
                 lambda: norm.checkpoint_weight_grad(x, x)):
        with pytest.raises(TypeError, match="CUDA/HIP"):
            call()




def layout(t, **kw):
    fake = torch.Tensor._make_subclass(_OnDevice, t)
    return norm._pitch(fake, "x", **kw)


class _OnDevice(torch.Tensor):
    is_cuda = True


def test_row_layouts():
    full = torch.zeros(6, 5, 40)
    assert layout(full) == (30, 40, 40)
    assert layout(full[..., :33]) == (30, 33, 40)
    assert layout(full[:, :, 7:]) == (30, 33, 40)
    assert layout(full[:, 2, :8]) == (6, 8, 200)
    assert layout(full[0, 0]) == (1, 40, 40)
    assert layout(full[:1, 3:4, :9]) == (1, 9, 9)
    assert layout(full[..., :0]) == (0, 0, 0)
    assert layout(full[:0, :, :8]) == (0, 8, 8)
    for bad in (full[:, :4, :8],                     # rows 40 apart, then 80
                full.transpose(1, 2), full[..., ::2],
                torch.zeros(1, 40).expand(6, 40)):
        with pytest.raises(ValueError):
            layout(bad)
    with pytest.raises(TypeError):
        layout(full.double())
    with pytest.raises(TypeError):
        layout(full, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        layout(torch.zeros(()))


def test_parameter_types():
    bf, f32 = torch.bfloat16, torch.float32
    w, b = torch.ones(4, dtype=bf), torch.ones(4)
    assert norm._param_type(None, None, bf) == bf and norm._param_type(None, b, bf) == f32
    with pytest.raises(TypeError, match="one type"):
        norm._param_type(w, b, bf)
    fake = torch.Tensor._make_subclass(_OnDevice, torch.ones(4, dtype=torch.float16))
    with pytest.raises(TypeError):
        norm._param(fake, 4, bf, "weight")
    fake = torch.Tensor._make_subclass(_OnDevice, torch.ones(4))
    with pytest.raises(ValueError):
        norm._param(fake, 5, bf, "weight")


def test_norm_linear_refuses_float32():
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        norm.norm_linear(torch.zeros(2, 8), None, None, torch.zeros(3, 8))
