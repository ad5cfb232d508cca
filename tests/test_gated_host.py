"""libtaco_gated without a GPU: its C ABI refuses every bad argument before
touching the device, and the torch layer refuses what it cannot pass on."""
import os
import re
import subprocess

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
if torch.cuda.device_count() > 0:
    # Fake device pointers below: only where no kernel could run on them.
    pytest.skip("host-only validation tests (fake device pointers)", allow_module_level=True)
gated = pytest.importorskip("gradients_taco_compress_amd.gated")

HEADER = os.path.join(ROOT, "include", "taco_gated.h")
OK, NULL, SHAPE, BLOCK, PARAM, ALIGN, ALIAS, HIP, FORMAT = range(9)
BF16, F16, F32 = range(3)
A = 1 << 24          # spacing of fake, aligned device addresses
WIDE = 1 << 20


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(taco_gated_[a-z0-9_]+)\s*\(", text)))


def test_every_declared_function_is_exported_and_bound():
    out = subprocess.run(["nm", "-D", "--defined-only", gated.LIB_PATH], capture_output=True,
                         text=True).stdout
    assert set(re.findall(r" T (taco_\w+)", out)) == set(declared()) == set(gated.EXPORTS)
    for n in declared():
        assert callable(getattr(gated, n))


def test_gated_sources_compile_like_the_rest(monkeypatch, tmp_path):
    import __graft_entry__ as g
    m = g._load_hip_build()
    cmds = []

    def fake_run(cmd, verbose):
        cmds.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
    monkeypatch.setattr(m, "_run", fake_run)
    monkeypatch.setattr(m, "GATED_LIB", str(tmp_path / "libtaco_gated.so"))
    monkeypatch.setattr(m, "GATED_TORCH", str(tmp_path / "_gated_torch.so"))
    m.build_gated()
    compiles = [c for c in cmds if "-c" in c]
    assert sorted(c[c.index("-c") + 1] for c in compiles) == sorted(m.GATED_SOURCES)
    feature = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    for c in compiles:
        assert "--offload-arch=gfx950" in c and "-O3" in c
        assert any(c[i:i + 4] == feature for i in range(len(c) - 3))
    assert not [f for f in os.listdir(m.CSRC) if ".tmp" in f]


def forward(x=A, ldx=64, wg=2 * A, ldg=64, wu=3 * A, ldu=64, rows=32, hidden=64, features=40,
            dtype=BF16, act=0, a=4 * A, lda=40, gate=0, up=0, ldgu=40, ws=7 * A, nbytes=None):
    if nbytes is None:
        nbytes = gated.taco_gated_forward_workspace(x, ldx, wg, ldg, wu, ldu, rows, hidden, features)
    return gated.taco_gated_forward(x, ldx, wg, ldg, wu, ldu, rows, hidden, features, dtype, act, a,
                                    lda, gate, up, ldgu, ws, nbytes, 0)


@pytest.mark.parametrize("rows", [4, 32, 96])
def test_forward_refusals(rows):
    def call(**kw):
        return forward(rows=kw.pop("rows", rows), **kw)
    assert call(dtype=F32) == FORMAT and call(dtype=-1) == FORMAT and call(dtype=3) == FORMAT
    assert call(rows=-1) == SHAPE and call(hidden=0, ldx=0) == SHAPE and call(features=0) == SHAPE
    assert call(hidden=WIDE + 1) == SHAPE and call(features=WIDE + 1) == SHAPE
    for name in ("ldx", "ldg", "ldu"):
        assert call(**{name: 63}) == SHAPE, name
    assert call(lda=39) == SHAPE and call(gate=5 * A, up=6 * A, ldgu=39) == SHAPE
    assert call(ldx=1 << 50) == SHAPE
    assert call(rows=1 << 40) == SHAPE                             # past any memory
    assert call(act=3) == PARAM and call(act=-1) == PARAM
    for name in ("x", "wg", "wu", "a"):
        assert call(**{name: 0}) == NULL, name
    assert call(gate=5 * A) == NULL and call(up=5 * A) == NULL      # both or neither
    for name, p in (("x", A), ("wg", 2 * A), ("wu", 3 * A), ("a", 4 * A)):
        assert call(**{name: p + 1}) == ALIGN, name
    assert call(gate=5 * A + 1, up=6 * A) == ALIGN
    assert call(a=A + 64) == ALIAS and call(a=2 * A) == ALIAS       # over x, over a weight
    assert call(gate=4 * A + 16, up=6 * A) == ALIAS and call(gate=5 * A, up=5 * A) == ALIAS
    assert call(rows=0, x=0, wg=0, wu=0, a=0) == OK
    # columns of one wider tensor do not overlap
    assert call(x=A, ldx=128, a=A + 128, lda=128, wg=A) == ALIAS


def test_forward_workspace():
    f = gated.taco_gated_forward_workspace

    def need(x=A, ldx=64, wg=2 * A, ldg=64, wu=3 * A, ldu=64, rows=96, hidden=64, features=40):
        return f(x, ldx, wg, ldg, wu, ldu, rows, hidden, features)
    assert need() == 0 and need(rows=0) == 0
    assert need(rows=-1) == need(hidden=0) == need(features=0) == need(ldx=63) == -1
    # operands that are not on 16-byte rows are copied; both weights, to one pitch
    assert need(x=A + 2) == 96 * 128
    assert need(ldx=65) == 96 * 128
    assert need(hidden=60) == 96 * 128 + 2 * 40 * 128
    assert need(wg=2 * A + 2) == 2 * 40 * 128
    assert need(ldg=72) == 2 * 40 * 128
    assert need(ldg=72, ldu=72) == 0
    assert need(ldx=1 << 23) == 96 * 128                             # too far apart to load in place
    # few rows read operands as they are: up to 16, and more where tiles would take longer
    wide = dict(hidden=16384, features=24, ldx=16384, ldg=16384, ldu=16384)
    assert need(rows=16, x=A + 2, hidden=60, ldg=72) == 0 and need(rows=16, x=A + 2, **wide) == 0
    assert need(rows=17, x=A + 2, hidden=60, ldg=72) == need(rows=64, x=A + 2, hidden=60, ldg=72) == 0
    assert need(rows=65, x=A + 2) == 65 * 128
    assert need(rows=17, **wide) > 0 and need(rows=64, **wide) > 0   # parts of a split
    # a long sum over few tiles is split
    split = need(ldx=WIDE, ldg=WIDE, ldu=WIDE, hidden=WIDE)
    assert split > 0 and split % (128 * 128 * 4) == 0
    assert forward(rows=96, x=A + 2, nbytes=96 * 128 - 1) == PARAM
    assert forward(rows=96, x=A + 2, ws=0) == NULL
    assert forward(rows=96, x=A + 2, ws=7 * A + 8) == ALIGN
    assert forward(rows=96, x=A + 2, ws=2 * A) == ALIAS


def backward(da=A, ldda=40, x=2 * A, ldx=64, gate=3 * A, up=4 * A, ldgu=40, wg=5 * A, ldg=64,
             wu=6 * A, ldu=64, rows=32, hidden=64, features=40, dtype=BF16, act=0, dx=7 * A, lddx=64,
             dg=8 * A, du=9 * A, ws=10 * A, nbytes=None):
    if nbytes is None:
        nbytes = gated.taco_gated_backward_workspace(x, ldx, wg, ldg, wu, ldu, rows, hidden, features,
                                                     int(dx != 0), int(dg != 0 or du != 0))
    return gated.taco_gated_backward(da, ldda, x, ldx, gate, up, ldgu, wg, ldg, wu, ldu, rows, hidden,
                                     features, dtype, act, dx, lddx, dg, du, ws, nbytes, 0)


def test_sizes_past_a_launch_are_refused():
    # 2^24 tiles of 128x64 outputs would take 2^32 threads
    f, b = gated.taco_gated_forward_workspace, gated.taco_gated_backward_workspace
    rows = 1 << 30
    assert f(A, 64, A, 64, A, 64, rows, 64, 64) >= 0
    assert f(A, 64, A, 64, A, 64, 2 * rows, 64, 64) == -1
    assert f(A, 128, A, 128, A, 128, rows, 128, 64) == -1
    assert f(A, 64, A, 64, A, 64, rows, 64, 128) == -1
    assert b(A, 64, A, 64, A, 64, 2 * rows, 64, 64, 1, 1) == -1
    assert gated.taco_gated_forward_mx_workspace(2 * rows, 64, 64) == -1
    assert f(A, WIDE, A, WIDE, A, WIDE, 32, WIDE, 65000) >= 0
    assert f(A, WIDE, A, WIDE, A, WIDE, 32, WIDE, 65536) == -1
    assert forward(rows=2 * rows, hidden=64, features=64, nbytes=0) == SHAPE


def test_backward_refusals():
    assert backward(dtype=F32) == FORMAT
    assert backward(rows=-1) == SHAPE and backward(ldda=39) == SHAPE and backward(ldgu=39) == SHAPE
    assert backward(ldx=63) == SHAPE and backward(lddx=63) == SHAPE and backward(ldu=63) == SHAPE
    assert backward(act=9) == PARAM
    for name in ("da", "x", "gate", "up", "wg", "wu", "ws"):
        assert backward(**{name: 0}) == NULL, name
    assert backward(dg=0) == NULL and backward(du=0) == NULL         # both or neither
    for name, n in (("da", 1), ("x", 2), ("gate", 3), ("up", 4), ("wg", 5), ("wu", 6), ("dx", 7),
                    ("dg", 8), ("du", 9)):
        assert backward(**{name: n * A + 1}) == ALIGN, name
    assert backward(ws=10 * A + 8) == ALIGN
    assert backward(dx=2 * A) == ALIAS and backward(dg=5 * A) == ALIAS and backward(du=8 * A) == ALIAS
    assert backward(ws=3 * A) == ALIAS
    need = gated.taco_gated_backward_workspace(2 * A, 64, 5 * A, 64, 6 * A, 64, 32, 64, 40, 1, 1)
    assert need >= 2 * 32 * 40 * 2 and backward(nbytes=need - 1) == PARAM
    # what only an output that is not asked for needs
    assert backward(dx=0, wg=0, wu=0, ldg=0, ldu=0, lddx=0, ws=0) == NULL     # the workspace only
    assert backward(dg=0, du=0, x=0, ldx=0, ws=0) == NULL
    assert backward(dx=0, dg=0, du=0, da=0, ws=0) == OK
    # no rows: weights' gradients are zeros, and have to be real for that
    assert backward(rows=0, dg=0, du=0) == OK
    assert backward(rows=0, dg=8 * A + 1) == ALIGN and backward(rows=0, du=8 * A) == ALIAS


def test_backward_workspace():
    f = gated.taco_gated_backward_workspace

    def need(x=A, ldx=64, wg=2 * A, ldg=64, wu=3 * A, ldu=64, rows=32, hidden=64, features=40, dx=1,
             dw=1):
        return f(x, ldx, wg, ldg, wu, ldu, rows, hidden, features, dx, dw)
    base = 2 * 32 * 40 * 2                                             # dG and dU
    assert need() == need(dx=0) == need(dw=0) == base
    assert need(dx=0, dw=0) == 0 and need(rows=0) == 0
    assert need(features=37) == base                                   # rows of 40
    assert need(x=A + 2) == base + 32 * 128 and need(x=A + 2, dw=0) == base
    assert need(wg=2 * A + 2) == base + 2 * 40 * 128 and need(wg=2 * A + 2, dx=0) == base
    assert need(rows=-1) == need(hidden=0) == need(ldx=63) == need(ldg=63) == -1
    assert need(ldx=63, dw=0) == need(ldg=63, dx=0) == base


def forward_mx(xc=A, xs=2 * A, gc=3 * A, gs=4 * A, uc=5 * A, us=6 * A, rows=32, hidden=64, features=40,
               dtype=BF16, act=0, a=7 * A, lda=40, ws=8 * A, nbytes=None):
    if nbytes is None:
        nbytes = gated.taco_gated_forward_mx_workspace(rows, hidden, features)
    return gated.taco_gated_forward_mx(xc, xs, gc, gs, uc, us, rows, hidden, features, dtype, act, a,
                                       lda, ws, nbytes, 0)


@pytest.mark.parametrize("rows", [4, 32, 96])
def test_forward_mx_refusals(rows):
    def call(**kw):
        return forward_mx(rows=kw.pop("rows", rows), **kw)
    assert call(dtype=F32) == FORMAT
    assert call(rows=-1) == SHAPE and call(hidden=48) == SHAPE and call(hidden=0) == SHAPE
    assert call(features=0) == SHAPE and call(lda=39) == SHAPE
    assert call(act=4) == PARAM
    for name in ("xc", "xs", "gc", "gs", "uc", "us", "a"):
        assert call(**{name: 0}) == NULL, name
    for name, n in (("xc", 1), ("gc", 3), ("uc", 5)):
        assert call(**{name: n * A + 8}) == ALIGN, name
    assert call(a=7 * A + 1) == ALIGN
    for n in range(1, 7):
        assert call(a=n * A) == ALIAS, n
    assert call(rows=0, xc=0, xs=0, gc=0, gs=0, uc=0, us=0, a=0) == OK


def test_forward_mx_workspace():
    f = gated.taco_gated_forward_mx_workspace
    assert f(16, 64, 40) == 0 and f(0, 64, 40) == 0 and f(64, 64, 40) == 0
    # scales by K-tile of 128 codes and 64 rows: 256 bytes each
    assert f(96, 64, 40) == 2 * 256 + 2 * 256
    assert f(65, 160, 130) == 2 * 2 * 256 + 2 * 2 * 3 * 256
    assert f(64, 16384, 24) > 128 * 3 * 256                          # and parts of a split
    assert f(-1, 64, 40) == f(32, 40, 40) == f(32, 64, 0) == -1
    need = f(96, 64, 40)
    assert forward_mx(rows=96, nbytes=need - 1) == PARAM
    assert forward_mx(rows=96, ws=0) == NULL and forward_mx(rows=96, ws=8 * A + 4) == ALIGN
    assert forward_mx(rows=96, ws=A) == ALIAS


def encode(x=A, ldx=64, rows=4, hidden=64, dtype=BF16, codes=2 * A, scales=3 * A):
    return gated.taco_gated_mx_encode(x, ldx, rows, hidden, dtype, codes, scales, 0)


def test_mx_encode_refusals():
    assert encode(dtype=3) == FORMAT
    assert encode(hidden=48) == SHAPE and encode(hidden=0) == SHAPE and encode(ldx=63) == SHAPE
    assert encode(rows=-1) == SHAPE and encode(hidden=2 * WIDE, ldx=2 * WIDE) == SHAPE
    for name in ("x", "codes", "scales"):
        assert encode(**{name: 0}) == NULL, name
    assert encode(x=A + 1) == ALIGN and encode(x=A + 2, dtype=F32) == ALIGN
    assert encode(codes=A) == ALIAS and encode(scales=2 * A + 100) == ALIAS
    assert encode(rows=0, x=0, codes=0, scales=0) == OK


def test_torch_layer_refuses_host_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(40, 64, dtype=torch.bfloat16)
    a = torch.zeros(4, 40, dtype=torch.bfloat16)
    c = (torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    for call in (lambda: gated.gated_forward(x, w, w),
                 lambda: gated.gated_backward(a, x, a, a, w, w),
                 lambda: gated.gated_forward_mx(c, c, c), lambda: gated.mx_encode(x)):
        with pytest.raises(TypeError, match="CUDA/HIP"):
            call()
    with pytest.raises(ValueError, match="silu"):
        gated.gated_forward_mx(c, c, c, "swish")
    with pytest.raises(TypeError, match="pair"):
        gated._mx(x, "x")


def test_feature_order_and_scale_tiles():
    """The order in which a half's rows hold features, and where a K-tile's scales
    lie, against the lanes that read them: of 32 features, lane group q's fragment
    j holds 8 q + 4 j + (0..3), so the two fragments of a lane are eight neighbours."""
    def feature_of_row(r):
        return (r & ~31) | (((r >> 2) & 3) << 3) | (((r >> 4) & 1) << 2) | (r & 3)
    assert sorted(feature_of_row(r) for r in range(128)) == list(range(128))
    for wave in range(4):
        for q in range(4):
            got = [feature_of_row(32 * wave + 16 * j + 4 * q + e) for j in range(2) for e in range(4)]
            assert got == [32 * wave + 8 * q + i for i in range(8)]
    src = open(os.path.join(ROOT, "gradients_taco_compress_amd", "csrc",
                            "taco_gated_internal.hpp")).read()
    assert "return (R & ~31) | (((R >> 2) & 3) << 3) | (((R >> 4) & 1) << 2) | (R & 3);" in src
