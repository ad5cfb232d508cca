"""Root-mean-square norm without a GPU: the C ABI refuses every bad argument
before touching the device."""
import os
import re
import subprocess

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
if torch.cuda.device_count() > 0:
    # Fake device pointers below: only where no kernel could run on them.
    pytest.skip("host-only validation tests (fake device pointers)", allow_module_level=True)
norm = pytest.importorskip("gradients_taco_compress_amd.norm")

OK, NULL, SHAPE, BLOCK, PARAM, ALIGN, ALIAS, HIP, FORMAT = range(9)
BF16, F16, F32 = range(3)
A = 1 << 24          # spacing of fake, aligned device addresses


def declared():
    text = open(os.path.join(ROOT, "include", "taco_rms.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(taco_rms_[a-z0-9_]+)\s*\(", text)))


def test_every_declared_function_is_exported_and_bound():
    out = subprocess.run(["nm", "-D", "--defined-only", norm.RMS_LIB_PATH], capture_output=True,
                         text=True).stdout
    assert set(re.findall(r" T (taco_\w+)", out)) == set(declared()) == set(norm.RMS_EXPORTS)
    for n in declared():
        assert callable(getattr(norm, n))


def test_rms_sources_compile_like_the_rest(monkeypatch, tmp_path):
    import __graft_entry__ as g
    m = g._load_hip_build()
    cmds = []

    def fake_run(cmd, verbose):
        cmds.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
    monkeypatch.setattr(m, "_run", fake_run)
    monkeypatch.setattr(m, "RMS_LIB", str(tmp_path / "libtaco_rms.so"))
    monkeypatch.setattr(m, "RMS_TORCH", str(tmp_path / "_rms_torch.so"))
    m.build_rms()
    compiles = [c for c in cmds if "-c" in c]
    assert sorted(c[c.index("-c") + 1] for c in compiles) == sorted(m.RMS_SOURCES)
    feature = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    for c in compiles:
        assert "--offload-arch=gfx950" in c and "-O3" in c
        assert any(c[i:i + 4] == feature for i in range(len(c) - 3))
    assert not [f for f in os.listdir(m.CSRC) if ".tmp" in f]


def forward(x=A, ldx=64, r=2 * A, ldr=64, rows=4, hidden=64, dtype=BF16, w=3 * A, pdtype=F32, eps=1e-5,
            y=4 * A, ldy=64, total=5 * A, ldt=64, rstd=6 * A):
    return norm.taco_rms_forward(x, ldx, r, ldr, rows, hidden, dtype, w, pdtype, eps, y, ldy,
                                      total, ldt, rstd, 0)


def mx(x=A, ldx=64, r=2 * A, ldr=64, rows=4, hidden=64, dtype=BF16, w=3 * A, pdtype=F32, eps=1e-5,
       codes=4 * A, scales=7 * A, total=5 * A, ldt=64):
    return norm.taco_rms_mx(x, ldx, r, ldr, rows, hidden, dtype, w, pdtype, eps, codes, scales,
                                 total, ldt, 0)


@pytest.mark.parametrize("call", [forward, mx])
def test_forward_refusals(call):
    assert call(dtype=3) == FORMAT and call(dtype=-1) == FORMAT
    assert call(pdtype=F16) == FORMAT and call(dtype=F32, pdtype=BF16) == FORMAT
    assert call(hidden=0, ldx=0) == SHAPE and call(hidden=1 << 21) == SHAPE and call(rows=-1) == SHAPE
    assert call(ldx=63) == SHAPE and call(ldr=63) == SHAPE and call(ldt=63) == SHAPE
    assert call(ldx=1 << 50) == SHAPE
    for eps in (-1e-9, float("nan"), float("inf")):
        assert call(eps=eps) == PARAM
    assert call(r=0) == PARAM                                       # a total without a residual
    assert call(x=0) == NULL
    assert call(x=A + 1) == ALIGN and call(r=2 * A + 1) == ALIGN and call(total=5 * A + 1) == ALIGN
    assert call(w=3 * A + 2) == ALIGN
    assert call(total=A + 64) == ALIAS and call(total=2 * A + 2) == ALIAS
    assert call(total=A, ldt=72) == ALIAS                           # x's place, another pitch
    assert call(total=3 * A) == ALIAS and call(w=5 * A) == ALIAS
    assert call(total=4 * A) == ALIAS
    assert call(rows=0, x=0, r=0, total=0) == OK


def test_forward_outputs():
    assert forward(y=0) == NULL and forward(y=4 * A + 1) == ALIGN and forward(rstd=6 * A + 2) == ALIGN
    assert forward(ldy=63) == SHAPE and forward(rstd=4 * A + 16) == ALIAS
    assert forward(y=A + 2) == ALIAS and forward(y=A, ldy=72) == ALIAS
    assert forward(y=5 * A) == ALIAS                                # y and total in one place
    assert forward(y=A, total=A) == ALIAS                           # both in x's


def test_mx_outputs():
    assert mx(codes=0) == NULL and mx(scales=0) == NULL
    assert mx(hidden=48) == SHAPE
    assert mx(codes=A) == ALIAS and mx(scales=4 * A + 100) == ALIAS and mx(codes=5 * A) == ALIAS


def backward(dy=A, lddy=64, x=2 * A, ldx=64, rstd=3 * A, dt=4 * A, lddt=64, w=5 * A, rows=4, hidden=64,
             dtype=BF16, pdtype=F32, dx=6 * A, lddx=64, dw=7 * A, ws=8 * A, nbytes=None):
    nbytes = norm.taco_rms_backward_workspace(rows, hidden) if nbytes is None else nbytes
    return norm.taco_rms_backward(dy, lddy, x, ldx, rstd, dt, lddt, w, rows, hidden, dtype, pdtype,
                                       dx, lddx, dw, ws, nbytes, 0)


def test_backward_refusals():
    assert backward(dtype=7) == FORMAT and backward(pdtype=F16) == FORMAT
    assert backward(rows=-1, nbytes=0) == SHAPE
    for name in ("lddy", "ldx", "lddt", "lddx"):
        assert backward(**{name: 63}) == SHAPE, name
    for name in ("dy", "x", "rstd", "dx", "ws"):
        assert backward(**{name: 0}) == NULL, name
    assert backward(dy=A + 1) == ALIGN and backward(ws=8 * A + 8) == ALIGN
    assert backward(dw=7 * A + 2) == ALIGN and backward(rstd=3 * A + 1) == ALIGN
    assert backward(dt=4 * A + 1) == ALIGN
    assert backward(dx=A + 2) == ALIAS and backward(dx=4 * A + 2) == ALIAS     # shifted over dy, dtotal
    assert backward(dx=A, lddx=72) == ALIAS and backward(dx=2 * A) == ALIAS
    assert backward(dw=A) == ALIAS and backward(ws=4 * A) == ALIAS and backward(dw=6 * A) == ALIAS
    assert backward(ws=5 * A) == ALIAS
    need = norm.taco_rms_backward_workspace(4, 64)
    assert need == 64 * 4 and backward(nbytes=need - 1) == PARAM
    assert backward(rows=0, dw=0, dx=0, dy=0, x=0) == OK
    assert backward(rows=0, dw=7 * A + 1) == ALIGN and backward(rows=0, dw=5 * A) == ALIAS


def test_backward_workspace():
    f = norm.taco_rms_backward_workspace
    assert f(0, 64) == 0
    assert f(-1, 64) == f(4, 0) == f(4, 1048577) == f(1 << 47, 1 << 10) == -1
    assert f(129, 64) == 16 * 64 * 4                          # sixteen segments of the rows
    assert f(1, 2560) == 2560 * 4 and f(1 << 20, 2560) == 512 * 2560 * 4


def test_torch_layer_refuses_host_tensors():
    x = torch.zeros(4, 64)
    for call in (lambda: norm.rms_norm(x), lambda: norm.rms_norm_mx(x),
                 lambda: norm.rms_norm_backward(x, x, x[:, 0])):
        with pytest.raises(TypeError, match="CUDA/HIP"):
            call()
