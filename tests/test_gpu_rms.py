"""Root-mean-square norm, with the residual's addition and into 8 bits, on the
GPU against the formulas in 64 bits.

Bounds are derived per element: u = eps / 2 of a type is the largest relative
rounding error to it (U32 for float32); a float32 sum of n terms in any order is
off by at most n U32 times the sum of the terms' magnitudes, and the kernels add
at most 40 terms in a row (8 a chunk, 8 chunks, then pairwise), wide rows
hidden / 1024 more.  Every case prints its name before it touches the GPU.
"""
from __future__ import annotations

import pytest
import torch

from gated_reference import BF, F16, F32, U32, half_step, mx_decode, mx_encode, rounding, within

pytestmark = pytest.mark.gpu

TYPES = [(BF, F32), (BF, BF), (F16, F32), (F16, F16), (F32, F32)]
# Around every limit of the kernels: parts of a wave, waves and work-groups to a
# row, ragged last chunks, and rows too wide to hold.
WIDTHS = [1, 2, 7, 8, 9, 64, 127, 128, 130, 256, 257, 504, 512, 513, 1000, 1024, 1025, 1536, 2048, 2056,
          2560, 3584, 4096, 4099, 6144, 8192, 8200, 12288, 12289, 16384, 16385, 20000]
MX_WIDTHS = [32, 64, 96, 128, 160, 256, 288, 512, 544, 1024, 1120, 1536, 2560, 3584, 4096, 4128, 8192,
             12288, 16384, 16416, 20000]


@pytest.fixture(scope="module")
def norm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gradients_taco_compress_amd.norm as norm
    return norm


def announce(msg):
    print(f"[case] {msg}", flush=True)


def depth(hidden):
    return 72 + (hidden / 1024 + 20 if hidden > 16384 else 0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows_of(rows, hidden, dtype, seed, scale=1.0, shift=0.0, pitch=0, offset=0):
    n = rows * (hidden + pitch) + offset
    flat = torch.empty(n, device="cuda").normal_(shift, scale, generator=gen(seed)).to(dtype)
    return flat[offset:].as_strided((rows, hidden), (hidden + pitch, 1))


def weight_of(hidden, dtype, seed=7):
    return torch.empty(hidden, device="cuda").normal_(1.0, 0.3, generator=gen(seed)).to(dtype)


class Forward64:
    def __init__(self, x, weight, eps, residual=None):
        s = x.double() + (0 if residual is None else residual.double())
        n = s.shape[1]
        w = torch.ones(n, device="cuda", dtype=torch.float64) if weight is None else weight.double()
        self.s = s
        self.e_s = 0.0 if residual is None else U32 * s.abs()           # one float32 addition
        mean = (s * s).mean(1)
        self.rstd = (mean + eps).rsqrt()
        # squares of values off by U32, their products and sum; division, addition, root, division
        self.e_rstd = self.rstd * (U32 * 4 + 0.5 * U32 * (depth(n) + 4) * mean / (mean + eps))
        self.y = s * self.rstd[:, None] * w
        self.e_y = self.y.abs() * (self.e_rstd / self.rstd + 4 * U32)[:, None]


def check_forward(norm, x, w, residual, eps=1e-5):
    ref = Forward64(x, w, eps, residual)
    y, total, rstd = norm.rms_norm(x, w, eps, residual=residual)
    within(rstd, ref.rstd, ref.e_rstd, "rstd")
    within(y, ref.y, ref.e_y + rounding(ref.y.abs() + ref.e_y, x.dtype), "y")
    if residual is None:
        assert total is None
    else:
        # one float32 addition, rounded once
        assert torch.equal(total, (x.float() + residual.float()).to(x.dtype))
    return y, total, rstd


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("hidden", WIDTHS)
def test_forward(norm, hidden, dtype, ptype):
    rows = 5 if hidden > 16 else 37
    for res in (False, True):
        announce(f"forward {rows}x{hidden} {dtype} {ptype} residual {res}")
        x = rows_of(rows, hidden, dtype, hidden, 1.5, 0.3)
        r = rows_of(rows, hidden, dtype, hidden + 1) if res else None
        check_forward(norm, x, weight_of(hidden, ptype), r)


@pytest.mark.parametrize("rows,hidden", [(1, 2560), (3000, 96), (2049, 200), (1000, 1536), (9000, 512),
                                         (4100, 1024), (700, 12288)])
def test_forward_many_rows(norm, rows, hidden):
    announce(f"forward {rows}x{hidden}")
    x, r = rows_of(rows, hidden, BF, 11), rows_of(rows, hidden, BF, 12)
    check_forward(norm, x, weight_of(hidden, F32), r)
    check_forward(norm, x, None, None)


@pytest.mark.parametrize("pitch,offset", [(8, 0), (24, 8), (5, 0), (0, 1), (3, 3), (4, 2)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides(norm, dtype, pitch, offset):
    for hidden in (72, 1000, 2568, 17000):
        announce(f"strides {hidden} {dtype} {pitch} {offset}")
        x = rows_of(6, hidden, dtype, 1, 1.0, 0.0, pitch, offset)
        r = rows_of(6, hidden, dtype, 2, 1.0, 0.0, 0 if pitch == 8 else pitch + 8, 0)
        w = weight_of(hidden, F32)
        y, total, rstd = check_forward(norm, x, w, r)
        out, tot = (torch.full((6, hidden + 9), 7.0, device="cuda", dtype=dtype) for _ in range(2))
        norm.rms_norm(x, w, 1e-5, residual=r, out=out[:, 4:4 + hidden], total=tot[:, 1:1 + hidden])
        assert torch.equal(out[:, 4:4 + hidden], y) and torch.equal(tot[:, 1:1 + hidden], total)
        out[:, 4:4 + hidden], tot[:, 1:1 + hidden] = 7.0, 7.0
        assert bool((out == 7.0).all()) and bool((tot == 7.0).all())
        dy = rows_of(6, hidden, dtype, 3, 1.0, 0.0, pitch, offset)
        check_backward(norm, dy, x, rstd, w, r)


@pytest.mark.parametrize("hidden", [40, 1111, 2560, 9000, 17000])
def test_in_place(norm, hidden):
    announce(f"in place {hidden}")
    x, r, w = rows_of(9, hidden, BF, 1), rows_of(9, hidden, BF, 2), weight_of(hidden, F32)
    y, total, rstd = norm.rms_norm(x, w, residual=r)
    for out_is, total_is in (("x", "r"), ("r", "x"), (None, "r"), ("x", None), (None, "x")):
        xs, rs = x.clone(), r.clone()
        place = {"x": xs, "r": rs, None: None}
        y2, t2, q2 = norm.rms_norm(xs, w, residual=rs, out=place[out_is], total=place[total_is])
        assert torch.equal(y2, y) and torch.equal(t2, total) and torch.equal(q2, rstd)
    xs = x.clone()
    assert torch.equal(norm.rms_norm(xs, w, out=xs)[0], norm.rms_norm(x, w)[0])
    dy = rows_of(9, hidden, BF, 3)
    dx, dw = norm.rms_norm_backward(dy, total, rstd, w, dtotal=r)
    for name in ("dy", "dtotal"):
        a, b = dy.clone(), r.clone()
        dx2, dw2 = norm.rms_norm_backward(a, total, rstd, w, dtotal=b, dx=a if name == "dy" else b)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    if hidden % 32 == 0:
        codes, scales, total = norm.rms_norm_mx(x, w, residual=r)
        xs, rs = x.clone(), r.clone()
        c2, s2, t2 = norm.rms_norm_mx(xs, w, residual=rs, total=rs)
        assert torch.equal(c2, codes) and torch.equal(s2, scales) and torch.equal(rs, total)


@pytest.mark.parametrize("hidden", [64, 2560, 16416])
def test_special_rows(norm, hidden):
    announce(f"special rows {hidden}")
    x = rows_of(7, hidden, F32, 1)
    x[0], x[1] = 0.0, 1e-30
    x[2] = 1e15
    x[3, 5], x[4, hidden - 1] = float("nan"), float("inf")
    y, _, rstd = norm.rms_norm(x, None, 1e-5)
    assert bool((y[0] == 0).all()) and abs(float(rstd[0]) - 1e-5 ** -0.5) < 1e-4
    assert bool(((y[2] - 1).abs() < 1e-5).all())
    assert bool(y[3].isnan().all()) and float(rstd[4]) == 0.0
    assert bool(y[4, hidden - 1].isnan()) and bool((y[4, :hidden - 1] == 0).all())
    clean = norm.rms_norm(rows_of(7, hidden, F32, 1), None, 1e-5)[0]
    assert torch.equal(y[5:], clean[5:])
    y, _, rstd = norm.rms_norm(x[:1], None, 0.0)               # 0 / 0
    assert bool(y.isnan().all()) and float(rstd) == float("inf")


def test_no_rows(norm):
    announce("no rows")
    x, w = rows_of(4, 64, BF, 1), weight_of(64, F32)
    y, total, rstd = norm.rms_norm(x[:0], w, residual=x[:0])
    assert y.shape == total.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = norm.rms_norm_backward(x[:0], x[:0], rstd, w)
    assert dx.shape == (0, 64) and dw.shape == (64,) and float(dw.abs().sum()) == 0.0
    codes, scales, total = norm.rms_norm_mx(x[:0], w)
    assert codes.shape == (0, 64) and scales.shape == (0, 2) and total is None


# ------------------------------------------------------------------ 8 bits --

@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("hidden", MX_WIDTHS)
def test_mx(norm, hidden, dtype, ptype):
    for res in (False, True):
        announce(f"mx {hidden} {dtype} {ptype} residual {res}")
        x = rows_of(9, hidden, dtype, hidden, 1.5)
        x[:, ::17] *= 20.0
        r = rows_of(9, hidden, dtype, 3) if res else None
        w = weight_of(hidden, ptype)
        ref = Forward64(x, w, 1e-5, r)
        codes, scales, total = norm.rms_norm_mx(x, w, 1e-5, residual=r)
        check_codes(codes, scales, ref)
        if res:
            assert torch.equal(total, (x.float() + r.float()).to(dtype))
        else:
            assert total is None


def check_codes(codes, scales, ref):
    """Codes and scales of y as the kernel has it, y off by at most ref.e_y: the
    maximum fits its scale and not half of it, and each code is nearest."""
    scale = torch.exp2(scales.double() - 127)
    top = ref.y.reshape(*scales.shape, 32).abs().amax(2)
    slack = ref.e_y.reshape(*scales.shape, 32).amax(2)
    assert bool((top - slack <= 448 * scale).all())
    assert bool((top + slack > 224 * scale).all())
    value = mx_decode(codes, scales)
    step = scale[..., None].expand(*scales.shape, 32).reshape(codes.shape)
    # E4M3: half a step is 2^-4 of the value, or 2^-10 of the scale below 2^-6 of it
    bound = torch.maximum(ref.y.abs() * 2.0 ** -4, step * 2.0 ** -10) + 2 * ref.e_y
    within(value, ref.y, bound, "codes")


@pytest.mark.parametrize("hidden", [32, 128, 1024, 2560, 4096, 16384, 17024])
def test_mx_codes_exactly(norm, hidden):
    """Rows of +-1 have q = 1 exactly, so y is the weight: any float32 numbers."""
    announce(f"mx exactly {hidden}")
    w = torch.empty(hidden, device="cuda").normal_(generator=gen(1))
    w *= torch.exp2(torch.randint(-30, 30, (hidden // 32,), generator=gen(2), device="cuda").float()
                    ).repeat_interleave(32)
    w[:32] = 0.0
    w[32:64] = torch.linspace(-448, 448, 32, device="cuda") if hidden > 32 else w[32:64]
    sign = torch.ones(3, hidden, device="cuda")
    sign[1] = -1.0
    sign[2, ::2] = -1.0
    want_codes, want_scales = mx_encode(sign * w)
    for dtype in (F32, BF, F16):
        codes, scales, _ = norm.rms_norm_mx(sign.to(dtype), w, 0.0)
        assert torch.equal(scales, want_scales), dtype
        assert torch.equal(codes, want_codes), dtype


@pytest.mark.parametrize("pitch,offset", [(8, 0), (5, 0), (0, 1), (3, 3)])
def test_mx_strides(norm, pitch, offset):
    for hidden in (96, 1120, 17024):
        announce(f"mx strides {hidden} {pitch} {offset}")
        x = rows_of(6, hidden, BF, 1, 1.0, 0.0, pitch, offset)
        r = rows_of(6, hidden, BF, 2, 1.0, 0.0, pitch + 8)
        got = norm.rms_norm_mx(x, None, residual=r)
        want = norm.rms_norm_mx(x.contiguous(), None, residual=r.contiguous())
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("hidden", [64, 2560, 16416])
def test_mx_of_rows_that_are_not_finite(norm, hidden):
    announce(f"mx nan {hidden}")
    x = rows_of(5, hidden, BF, 1)
    clean = norm.rms_norm_mx(x)
    x[1, 3], x[2, hidden - 1] = float("nan"), float("inf")
    codes, scales, _ = norm.rms_norm_mx(x)
    assert bool((codes[1] == 127).all()) and bool((scales[1] == 255).all())
    # q = 0: the infinity's block is NaN, the others are zeros
    assert bool((codes[2, -32:] == 127).all()) and int(scales[2, -1]) == 255
    assert bool((codes[2, :-32] == 0).all()) and bool((scales[2, :-1] == 0).all())
    for i in (0, 3, 4):
        assert torch.equal(codes[i], clean[0][i]) and torch.equal(scales[i], clean[1][i])


# ---------------------------------------------------------------- backward --

def check_backward(norm, dy, x, rstd, w, dtotal):
    n, rows = x.shape[1], x.shape[0]
    dyd, q = dy.double(), rstd.double()[:, None]
    h = x.double() * q
    wd = torch.ones(n, device="cuda", dtype=torch.float64) if w is None else w.double()
    g = dyd * wd
    mean = (g * h).mean(1, keepdim=True)
    e_mean = U32 * (depth(n) + 4) * (g * h).abs().mean(1, keepdim=True)
    dx = q * (g - h * mean)
    e_dx = q * (g.abs() * 3 * U32 + h.abs() * (e_mean + 4 * U32 * mean.abs())) + 2 * U32 * dx.abs()
    if dtotal is not None:
        dx = dx + dtotal.double()
        e_dx = e_dx + U32 * dx.abs()
    got, dw = norm.rms_norm_backward(dy, x, rstd, w, dtotal=dtotal)
    within(got, dx, e_dx + rounding(dx.abs() + e_dx, dy.dtype), "dx")
    want = (dyd * h).sum(0)
    e_dw = U32 * (rows + 40) * (dyd * h).abs().sum(0)
    ptype = F32 if w is None else w.dtype
    assert dw.dtype == ptype
    within(dw, want, e_dw + rounding(want.abs() + e_dw, ptype), "dweight")
    return got, dw


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("hidden", WIDTHS)
def test_backward(norm, hidden, dtype, ptype):
    rows = 5 if hidden > 16 else 37
    for res in (False, True):
        announce(f"backward {rows}x{hidden} {dtype} {ptype} dtotal {res}")
        x, dy = rows_of(rows, hidden, dtype, hidden, 1.5, 0.3), rows_of(rows, hidden, dtype, 5)
        rstd = (x.float() ** 2).mean(1).add(1e-5).rsqrt()
        check_backward(norm, dy, x, rstd, weight_of(hidden, ptype),
                       rows_of(rows, hidden, dtype, 6) if res else None)


@pytest.mark.parametrize("rows,hidden", [(3000, 96), (2049, 200), (1300, 1536), (9000, 512), (700, 12288),
                                         (600, 16384), (70, 17000), (20000, 64)])
def test_backward_many_rows(norm, rows, hidden):
    """Several rows to a work-group and a part of a turn; without a weight."""
    announce(f"backward {rows}x{hidden}")
    x, dy = rows_of(rows, hidden, BF, 1), rows_of(rows, hidden, BF, 2)
    rstd = (x.float() ** 2).mean(1).add(1e-5).rsqrt()
    check_backward(norm, dy, x, rstd, None, rows_of(rows, hidden, BF, 3))
    dx, dw = norm.rms_norm_backward(dy, x, rstd, None, param_dtype=BF)
    assert dw.dtype == BF
    only, none = norm.rms_norm_backward(dy, x, rstd, None, param_grads=False)
    assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,hidden", [(1, 8), (2, 63), (33, 65), (64, 1000), (200, 2567), (255, 130), (256, 4096),
                                         (257, 4080), (85, 12288), (86, 12288), (128, 1025), (129, 8), (129, 100), (129, 1024),
                                         (130, 1025), (511, 136), (512, 1000), (513, 1000), (2048, 128), (2048, 129),
                                         (2049, 128)])
def test_backward_of_few_rows(norm, rows, hidden, dtype):
    """Either side of where the weight's gradient is made beside dx, and in dy's
    place, where it is made before."""
    announce(f"backward, few rows {rows}x{hidden} {dtype}")
    x, dy, dt = (rows_of(rows, hidden, dtype, s) for s in (1, 2, 3))
    rstd, w = (x.float() ** 2).mean(1).add(1e-5).rsqrt(), weight_of(hidden, F32)
    dx, dw = check_backward(norm, dy, x, rstd, w, dt)
    into = dy.clone()
    dx2, dw2 = norm.rms_norm_backward(into, x, rstd, w, dtotal=dt, dx=into)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    only, none = norm.rms_norm_backward(dy, x, rstd, w, dtotal=dt, param_grads=False)
    assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("rows,hidden", [(1, 40), (64, 128), (1025, 128), (5000, 1000), (300, 17000)])
def test_weight_gradient_sums_are_exact(norm, rows, hidden):
    announce(f"exact sums {rows}x{hidden}")
    x = torch.randint(-2, 3, (rows, hidden), generator=gen(1), device="cuda").to(BF)
    dy = torch.randint(-2, 3, (rows, hidden), generator=gen(2), device="cuda").to(BF)
    rstd = torch.exp2(torch.randint(-1, 2, (rows,), generator=gen(3), device="cuda").float())
    _, dw = norm.rms_norm_backward(dy, x, rstd, None)
    assert torch.equal(dw.double(), (dy.double() * x.double() * rstd.double()[:, None]).sum(0))


def test_nan_stays_in_its_row_and_column(norm):
    announce("backward nan")
    x, dy = rows_of(300, 1000, BF, 1), rows_of(300, 1000, BF, 2)
    rstd = (x.float() ** 2).mean(1).add(1e-5).rsqrt()
    dx, dw = norm.rms_norm_backward(dy, x, rstd, None)
    dy[7, 11] = float("nan")
    dx2, dw2 = norm.rms_norm_backward(dy, x, rstd, None)
    assert bool(dx2[7].isnan().all()) and bool(dw2[11].isnan())
    keep = torch.arange(300, device="cuda") != 7
    assert torch.equal(dx2[keep], dx[keep])
    cols = torch.arange(1000, device="cuda") != 11
    assert torch.equal(dw2[cols], dw[cols])


def test_offsets_past_32_bits(norm):
    announce("offsets past 32 bits")
    rows, pitch = 9, 1 << 29
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB")
    full = torch.empty(rows * pitch, device="cuda", dtype=BF)
    x, out = full.as_strided((rows, 64), (pitch, 1)), full[4096:].as_strided((rows, 64), (pitch, 1))
    total = full[8192:].as_strided((rows, 64), (pitch, 1))
    small, r = rows_of(rows, 64, BF, 1), rows_of(rows, 64, BF, 2)
    x.copy_(small)
    want = norm.rms_norm(small, None, residual=r)
    norm.rms_norm(x, None, residual=r, out=out, total=total)
    assert torch.equal(out, want[0]) and torch.equal(total, want[1])
    dx, dw = norm.rms_norm_backward(small, want[1], want[2])
    dx2 = full[12288:].as_strided((rows, 64), (pitch, 1))
    _, dw2 = norm.rms_norm_backward(x, total, want[2], dx=dx2)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


# --------------------------------------------------- streams, graphs, repeat --

def test_another_stream_and_repeats(norm):
    announce("another stream")
    s = torch.cuda.Stream()
    x, r, w = rows_of(300, 1024, BF, 1), rows_of(300, 1024, BF, 2), weight_of(1024, F32)
    dy = rows_of(300, 1024, BF, 3)

    def all_of(**kw):
        y, total, rstd = norm.rms_norm(x, w, residual=r, **kw)
        return (y, total, rstd, *norm.rms_norm_mx(x, w, residual=r, **kw)[:2],
                *norm.rms_norm_backward(dy, total, rstd, w, dtotal=r, **kw))
    want = all_of()
    torch.cuda.synchronize()
    got = all_of(stream=s)
    with torch.cuda.stream(s):
        inside = all_of()
    s.synchronize()
    for other in (got, inside, all_of()):
        assert all(torch.equal(p, q) for p, q in zip(other, want))


def test_graph_replays(norm):
    announce("graph")
    x, r, w = rows_of(70, 1111, BF, 1), rows_of(70, 1111, BF, 2), weight_of(1111, F32)
    dy = rows_of(70, 1111, BF, 3)

    def step():
        y, total, rstd = norm.rms_norm(x, w, residual=r)
        codes, scales, _ = norm.rms_norm_mx(x[:, :1088], None)
        return (y, total, rstd, codes, scales, *norm.rms_norm_backward(dy, total, rstd, w, dtotal=r))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for turn in range(4):
        x.copy_(rows_of(70, 1111, BF, 30 + turn))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        assert all(torch.equal(p, q) for p, q in zip(got, step())), turn


# ---------------------------------------------------------------- autograd --

def plain(x, w, eps, r):
    s = x if r is None else x + r
    y = s * (s * s).mean(-1, keepdim=True).add(eps).rsqrt()
    return (y if w is None else y * w), s


@pytest.mark.parametrize("ptype", [F32, None])
@pytest.mark.parametrize("use", ["y", "total", "both", "no residual"])
def test_autograd_against_64_bits(norm, use, ptype):
    announce(f"autograd {use} {ptype}")
    x, r = rows_of(6, 200, F32, 1).view(2, 3, 200), rows_of(6, 200, F32, 2).view(2, 3, 200)
    w = None if ptype is None else weight_of(200, ptype)
    dy, dt = rows_of(6, 200, F32, 3).view(2, 3, 200), rows_of(6, 200, F32, 4).view(2, 3, 200)
    res = use != "no residual"
    leaves = [t.clone().requires_grad_() for t in ([x, r] if res else [x]) + ([] if w is None else [w])]
    exact = [t.detach().double().requires_grad_() for t in leaves]

    def run(fn, ts, cast):
        ww = None if w is None else ts[-1]
        out = fn(ts[0], ww, 1e-5, ts[1] if res else None)
        y, total = out if isinstance(out, tuple) else (out, None)
        loss = 0
        if use != "total":
            loss = loss + (y * cast(dy)).sum()
        if res and use in ("total", "both"):
            loss = loss + (total * cast(dt)).sum()
        loss.backward()
    run(lambda a, b, c, d: norm.rms(a, b, c, residual=d), leaves, lambda t: t)
    run(plain, exact, lambda t: t.double())
    for got, want in zip(leaves, exact):
        if want.grad is None:
            assert got.grad is None or float(got.grad.abs().sum()) == 0
            continue
        assert got.grad.shape == got.shape and got.grad.dtype == got.dtype
        # sums of 200 float32 terms, a few roundings: far below 1e-5 of the gradient's size
        assert float((got.grad.double() - want.grad).norm() / want.grad.norm()) < 1e-5


def test_autograd_gradients_are_differences(norm):
    announce("differences")
    x, r, w = rows_of(3, 40, F32, 1), rows_of(3, 40, F32, 2), weight_of(40, F32)
    dy, dt = rows_of(3, 40, F32, 3).double(), rows_of(3, 40, F32, 4).double()
    leaves = [t.clone().requires_grad_() for t in (x, r, w)]
    y, total = norm.rms(leaves[0], leaves[2], 1e-5, residual=leaves[1])
    torch.autograd.backward([y, total], [dy.float(), dt.float()])

    def loss(a, b, c):
        y, total, _ = norm.rms_norm(a, c, 1e-5, residual=b)
        return float((y.double() * dy).sum() + (total.double() * dt).sum())
    for i, leaf in enumerate(leaves):
        g = leaf.grad.double()
        h = 1e-2 * float(leaf.detach().double().norm() / g.norm())
        args = [x, r, w]
        args[i] = (args[i].double() + h * g).float()
        up = loss(*args)
        args = [x, r, w]
        args[i] = (args[i].double() - h * g).float()
        # third-order terms: 1e-4 of the size, times a few
        want = 2 * h * float((g * g).sum())
        assert abs(up - loss(*args) - want) < 2e-3 * want


def test_a_training_step_with_the_gated_block(norm):
    """x, r -> norm with the residual -> gated block -> linear, and back, in bf16,
    against the same in 64 bits."""
    announce("training step")
    from gradients_taco_compress_amd import gated
    rows, hidden, features = 200, 96, 160
    x, r = rows_of(rows, hidden, BF, 1), rows_of(rows, hidden, BF, 2)
    wn = weight_of(hidden, F32)
    wg, wu = (rows_of(features, hidden, BF, 3 + i, hidden ** -0.5) for i in range(2))
    wd = rows_of(hidden, features, BF, 5, features ** -0.5)
    dout = rows_of(rows, hidden, BF, 6)
    leaves = [t.clone().requires_grad_() for t in (x, r, wn, wg, wu, wd)]
    y, total = norm.rms(leaves[0], leaves[2], residual=leaves[1])
    out = total + torch.nn.functional.linear(gated.gated(y, leaves[3], leaves[4]), leaves[5])
    out.backward(dout)
    exact = [t.detach().double().requires_grad_() for t in leaves]
    yd, td = plain(exact[0], exact[2], 1e-5, exact[1])
    od = td + (torch.nn.functional.silu(yd @ exact[3].t()) * (yd @ exact[4].t())) @ exact[5].t()
    od.backward(dout.double())

    def off(a, b):
        return float((a.detach().double() - b.detach()).norm() / b.detach().norm())
    # Roundings to bf16 on the way (total, y, G, U, A, the linear layer's result, out, and as
    # many back), each at most half a step of terms of the result's own size.
    assert off(out, od) < 8 * half_step(BF)
    for got, want in zip(leaves, exact):
        assert off(got.grad, want.grad) < 12 * half_step(BF)


def test_residual_of_other_leading_dimensions(norm):
    announce("residual's shape")
    x, r = rows_of(6, 200, BF, 1), rows_of(6, 200, BF, 2)
    w, dy, dt = weight_of(200, BF), rows_of(6, 200, BF, 3), rows_of(6, 200, BF, 4)
    same = [t.clone().requires_grad_() for t in (x, r, w)]
    torch.autograd.backward(norm.rms(same[0], same[2], residual=same[1]), (dy, dt))
    for use_y in (True, False):
        leaves = [x.view(2, 3, 200).clone().requires_grad_(), r.clone().requires_grad_(),
                  w.clone().requires_grad_()]
        y, total = norm.rms(leaves[0], leaves[2], residual=leaves[1])
        assert y.shape == total.shape == leaves[0].shape
        if use_y:
            torch.autograd.backward((y, total), (dy.view(2, 3, 200), dt.view(2, 3, 200)))
        else:
            total.backward(dt.view(2, 3, 200))
        for i in (0, 1):
            assert torch.equal(leaves[i].grad.view(6, 200), same[i].grad if use_y else dt)


def test_the_sum_of_a_tensor_with_itself(norm):
    announce("x twice")
    x, w, dy = rows_of(5, 96, F32, 1), weight_of(96, F32), rows_of(5, 96, F32, 3)
    a, exact = x.clone().requires_grad_(), x.double().requires_grad_()
    norm.rms(a, w, residual=a)[0].backward(dy)
    plain(exact, w.double(), 1e-5, exact)[0].backward(dy.double())
    assert float((a.grad.double() - exact.grad).norm() / exact.grad.norm()) < 1e-5


def test_a_captured_training_step(norm):
    """Forward and backward through autograd in one graph (no eager graph of the same
    leaves alive), replayed on new inputs with eager steps in between."""
    announce("captured step")
    from gradients_taco_compress_amd import gated
    rows, hidden, features = 70, 96, 40

    def fresh(seed):
        return [rows_of(rows, hidden, BF, seed), rows_of(rows, hidden, BF, seed + 1),
                weight_of(hidden, F32), rows_of(features, hidden, BF, 3, hidden ** -0.5),
                rows_of(features, hidden, BF, 4, hidden ** -0.5)]
    leaves = [t.requires_grad_() for t in fresh(10)]
    da, dt = rows_of(rows, features, BF, 8), rows_of(rows, hidden, BF, 9)

    def step(ts):
        for t in ts:
            t.grad = None
        y, total = norm.rms(ts[0], ts[2], residual=ts[1])
        a = gated.gated(y, ts[3], ts[4])
        torch.autograd.backward((a, total), (da, dt))
        return a.detach()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaves)
    for turn in range(4):
        new = fresh(20 + 5 * turn)
        with torch.no_grad():
            for t, v in zip(leaves, new):
                t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [out.clone()] + [t.grad.clone() for t in leaves]
        eager = [t.requires_grad_() for t in new]
        want = [step(eager)] + [t.grad for t in eager]
        assert all(torch.equal(p, q) for p, q in zip(got, want)), turn


def test_serving_in_8_bits(norm):
    """The norm's 8-bit rows into the gated block's 8-bit pass, against 64 bits on
    the same codes, and against the 16-bit pass within what 8 bits lose."""
    announce("serving")
    from gradients_taco_compress_amd import gated
    from gated_reference import Forward64 as Gated64, mx_dot_error
    for rows in (3, 40):
        x, r = rows_of(rows, 256, BF, 1), rows_of(rows, 256, BF, 2)
        w = weight_of(256, F32)
        wg, wu = (rows_of(96, 256, BF, 3 + i, 256 ** -0.5) for i in range(2))
        codes, scales, total = norm.rms_norm_mx(x, w, residual=r)
        pairs = [(codes, scales), gated.mx_encode(wg), gated.mx_encode(wu)]
        a = gated.gated_forward_mx(*pairs)
        d = [mx_decode(*p) for p in pairs]
        Gated64(*d, "silu", (mx_dot_error(d[0], d[1]), mx_dot_error(d[0], d[2]))).check(a)
        y, total16, _ = norm.rms_norm(x, w, residual=r)
        assert torch.equal(total, total16)
        b = gated.gated_forward(y, wg, wu)
        # each of four operands (x and a weight, in G and in U) is off by at most 2^-4 an element
        assert float((a.double() - b.double()).norm() / b.double().norm()) < 4 * 2.0 ** -4


# ---------------------------------------------------------------- refusals --

def test_refusals(norm):
    announce("refusals")
    x, w = rows_of(4, 64, BF, 1), weight_of(64, F32)
    with pytest.raises(TypeError, match="CUDA/HIP"):
        norm.rms_norm(x.cpu(), None)
    with pytest.raises(TypeError):
        norm.rms_norm(x.double(), None)
    for bad in (w[:63], w.half(), w.double()):
        with pytest.raises((TypeError, ValueError)):
            norm.rms_norm(x, bad)
    for bad in (x[:3], x.float(), x[:, :63]):
        with pytest.raises((TypeError, ValueError)):
            norm.rms_norm(x, w, residual=bad)
    with pytest.raises(ValueError, match="residual"):
        norm.rms_norm(x, w, total=torch.empty_like(x))
    with pytest.raises(ValueError, match="residual"):
        norm.rms_norm_mx(x, w, total=torch.empty_like(x))
    with pytest.raises(norm.TacoError, match="PARAM"):
        norm.rms_norm(x, w, -1.0)
    with pytest.raises(norm.TacoError, match="PARAM"):
        norm.rms_norm(x, w, float("nan"))
    with pytest.raises(ValueError, match="multiple of 32"):
        norm.rms_norm_mx(x[:, :48], w[:48])
    flat = torch.zeros(4 * 64 + 1, device="cuda", dtype=BF)
    with pytest.raises(norm.TacoError, match="ALIAS"):
        norm.rms_norm(flat[1:].view(4, 64), w, out=flat[:-1].view(4, 64))
    y = torch.empty_like(x)
    with pytest.raises(norm.TacoError, match="ALIAS"):
        norm.rms_norm(x, w, residual=x.clone(), out=y, total=y)
    _, _, rstd = norm.rms_norm(x, w)
    for args in ((x, x[:3], rstd), (x, x, rstd[:3]), (x, x.float(), rstd)):
        with pytest.raises((TypeError, ValueError)):
            norm.rms_norm_backward(*args, w)
    with pytest.raises(TypeError, match="param_dtype"):
        norm.rms_norm_backward(x, x, rstd, w, param_dtype=BF)
    with pytest.raises(norm.TacoError, match="ALIAS"):
        norm.rms_norm_backward(x, y, rstd, w, dx=y)
