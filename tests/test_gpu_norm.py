"""Layer norm and its 8-bit checkpoint on the GPU against the formulas in 64 bits.

Tolerances are derived, per element, from the roundings on the way: u = eps/2
of a type is the largest relative rounding error to it (U32 for float32).  A
float32 sum of n terms in any order is off by at most (n - 1) U32 times the
sum of the terms' magnitudes; the kernels add at most 40 terms in a row
(8 per chunk, 4 chunks, then pairwise), wide rows hidden / 1024 more.
Every case prints its name before it touches the GPU.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

U32 = torch.finfo(torch.float32).eps / 2
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF, F32), (BF, BF), (F16, F32), (F16, F16), (F32, F32)]
# Around every limit of the kernels: sub-wave and wave rows, one to four chunks
# per thread, ragged last chunks, and rows too wide to hold.
WIDTHS = [1, 2, 7, 8, 9, 64, 127, 128, 129, 130, 504, 512, 513, 1000, 1024, 1025, 1111, 2048,
          2056, 2560, 4096, 4099, 6144, 6152, 8192, 8200, 12288, 12289, 16384, 16385, 20000]


@pytest.fixture(scope="module")
def norm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gradients_taco_compress_amd.norm as norm
    return norm


def announce(msg):
    print(f"[case] {msg}", flush=True)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(v, dtype):
    """Largest error of rounding v to dtype (its smallest steps included)."""
    info = torch.finfo(dtype)
    return v.abs() * half_step(dtype) + info.tiny * info.eps


def depth(hidden):
    return 40 + (hidden / 1024 + 20 if hidden > 16384 else 0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows_of(rows, hidden, dtype, seed, scale=1.0, shift=0.0, pitch=0, offset=0):
    """[rows, hidden] of N(shift, scale), rows hidden + pitch elements apart,
    starting `offset` elements into its memory."""
    n = rows * (hidden + pitch) + offset
    flat = torch.empty(n, device="cuda").normal_(shift, scale, generator=gen(seed)).to(dtype)
    return flat[offset:].as_strided((rows, hidden), (hidden + pitch, 1))


def params(hidden, dtype, seed):
    w = torch.empty(hidden, device="cuda").normal_(1.0, 0.3, generator=gen(seed)).to(dtype)
    b = torch.empty(hidden, device="cuda").normal_(0.0, 0.5, generator=gen(seed + 1)).to(dtype)
    return w, b


class Forward64:
    """The forward formulas in 64 bits, with bounds on what float32 adds."""

    def __init__(self, x, weight, bias, eps):
        x = x.double()
        n = x.shape[1]
        d = depth(n)
        self.mean = x.mean(1)
        dev = x - self.mean[:, None]
        var = (dev * dev).mean(1)
        self.rstd = (var + eps).rsqrt()
        self.h = dev * self.rstd[:, None]
        w = torch.ones(n, device="cuda", dtype=torch.float64) if weight is None else weight.double()
        b = torch.zeros_like(w) if bias is None else bias.double()
        self.y = self.h * w + b
        # mean: the sum, the division.  var: deviations from a mean that is
        # off by e_mean (twice, since waves merge), their squares and sum.
        self.e_mean = U32 * (d + 2) * x.abs().mean(1)
        e_var = U32 * (d + 8) * var + 2 * self.e_mean * dev.abs().mean(1) + self.e_mean ** 2
        self.e_rstd = self.rstd * (U32 * 4 + 0.5 * e_var / (var + eps))
        self.e_h = (self.rstd[:, None] * (self.e_mean[:, None] + 2 * U32 * dev.abs())
                    + self.h.abs() * (self.e_rstd / self.rstd)[:, None])
        self.e_y = self.e_h * w.abs() + 2 * U32 * ((self.h * w).abs() + b.abs())


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {err.numel()} past the bound, worst "
                                 f"{float((err / bound)[bad].max()):.3g} times it")


def check_forward(norm, x, w, b, eps=1e-5):
    ref = Forward64(x, w, b, eps)
    y, mean, rstd = norm.layer_norm(x, w, b, eps)
    within(mean, ref.mean, ref.e_mean + 1e-30, "mean")
    within(rstd, ref.rstd, ref.e_rstd, "rstd")
    within(y, ref.y, ref.e_y + rounding(ref.y, x.dtype), "y")
    y2, codes, rstd2 = norm.layer_norm_checkpoint(x, w, b, eps)
    assert torch.equal(y2, y) and torch.equal(rstd2, rstd)
    s = norm.checkpoint_scale(x.shape[1])
    value = codes.view(torch.float8_e4m3fn).double()
    v = ref.h * s
    within(value, v, torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, device="cuda",
                                                                     dtype=torch.float64))
           + ref.e_h * s * (1 + 2.0 ** -3), "codes")


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("hidden", WIDTHS)
def test_forward(norm, hidden, dtype, ptype):
    rows = 5 if hidden > 16 else 37
    announce(f"forward {rows}x{hidden} {dtype} {ptype}")
    x = rows_of(rows, hidden, dtype, hidden, 1.5, 0.3)
    w, b = params(hidden, ptype, 7)
    check_forward(norm, x, w, b)


@pytest.mark.parametrize("rows,hidden", [(1, 2560), (3000, 96), (2049, 200), (1000, 1536),
                                         (4100, 1024), (700, 12288)])
def test_forward_many_rows(norm, rows, hidden):
    announce(f"forward {rows}x{hidden}")
    w, b = params(hidden, F32, 3)
    check_forward(norm, rows_of(rows, hidden, BF, 11), w, b)


@pytest.mark.parametrize("pitch,offset", [(8, 0), (24, 8), (5, 0), (0, 1), (3, 3), (4, 2)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_strides(norm, dtype, pitch, offset):
    for hidden in (72, 1000, 2568, 17000):
        announce(f"forward strides {hidden} {dtype} pitch {pitch} offset {offset}")
        x = rows_of(9, hidden, dtype, 5, pitch=pitch, offset=offset)
        w, b = params(hidden, F32, 9)
        check_forward(norm, x, w, b)
        # Into a wider buffer: what lies between the rows stays.
        out = rows_of(9, hidden, dtype, 6, pitch=pitch, offset=offset)
        base = out._base if out._base is not None else out
        before = base.clone()
        y, _, _ = norm.layer_norm(x, w, b, out=out)
        want, _, _ = norm.layer_norm(x.contiguous(), w, b)
        assert torch.equal(out, want)
        out.copy_(before.as_strided(out.shape, out.stride(), out.storage_offset()))
        assert torch.equal(base, before)


@pytest.mark.parametrize("hidden", [33, 1024, 4104, 20000])
def test_forward_without_parameters(norm, hidden):
    announce(f"forward without parameters {hidden}")
    x = rows_of(6, hidden, BF, 21)
    w, b = params(hidden, BF, 4)
    for weight, bias in ((None, None), (w, None), (None, b)):
        check_forward(norm, x, weight, bias)


@pytest.mark.parametrize("hidden", [8, 100, 512, 2560, 12288, 20000])
def test_special_rows(norm, hidden):
    """Constant rows, rows far from zero, one entry that holds all of a row's
    energy (the largest code), and rows with NaN or infinity among others."""
    announce(f"special rows {hidden}")
    x = rows_of(7, hidden, F32, 31)
    x[0] = 0.0
    x[1] = 3.25
    x[2] += 1000.0
    x[3] = 0.0
    x[3, hidden // 2] = 5.0e4
    w, b = params(hidden, F32, 5)
    check_forward(norm, x[:5], w, b)
    y, codes, rstd = norm.layer_norm_checkpoint(x[:2], w, b)
    assert torch.equal(y, b.expand(2, hidden)) and not codes.any()
    assert torch.allclose(rstd, torch.full((2,), 1e-5, device="cuda").rsqrt(), rtol=4 * U32)
    peak = norm.layer_norm_checkpoint(x[3:4], w, b)[1].view(torch.float8_e4m3fn).float().max()
    assert 100 <= float(peak) <= 448
    good = norm.layer_norm_checkpoint(x, w, b)
    x[5, hidden - 1] = float("inf")
    x[6, 0] = float("nan")
    bad = norm.layer_norm_checkpoint(x, w, b)
    for g, t in zip(good, bad):
        assert torch.equal(g[:5], t[:5])
    assert bad[0][5:].isnan().all() and ((bad[1][5:] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("hidden", [40, 520, 2560, 12288, 16392, 20000, 65537])
def test_rows_within_their_mean_s_rounding(norm, hidden):
    """float32 rows whose spread is at or below the rounding of their mean: h
    is made of rounding alone, yet its squares stay within the row's length,
    so no code overflows.  An element's squared deviation is at most twice
    what the merged sums hold of it, hence the factors of 1.5."""
    announce(f"rows within their mean's rounding {hidden}")
    values = torch.tensor([3.3, 1e6 / 3, 1e9 / 3, 1e9 / 7, 1e12 / 7, -2.2e9], device="cuda")
    x = values[:, None].expand(-1, hidden).contiguous()
    x = torch.cat([x, x])
    x[6:, hidden // 3] = torch.nextafter(values, values + values.abs())
    h, codes, rstd = norm.layer_norm_checkpoint(x, None, None)
    assert rstd.isfinite().all() and ((codes & 0x7F) != 0x7F).all()
    assert float(h[:6].abs().max()) <= 1.5
    assert float(h[6:].abs().max()) <= 1.5 * hidden ** 0.5


def test_eps_enters(norm):
    x = rows_of(4, 256, F32, 41, 1e-3)
    for eps in (0.0, 1e-12, 1e-2, 3.0):
        announce(f"eps {eps}")
        check_forward(norm, x, None, None, eps)


# ---------------------------------------------------------------- backward --

def backward64(dy, h, rstd, weight):
    """dx, dw, db in 64 bits, with the magnitudes that bound float32's errors."""
    dy, rstd = dy.double(), rstd.double()[:, None]
    n = dy.shape[1]
    w = torch.ones(n, device="cuda", dtype=torch.float64) if weight is None else weight.double()
    g = dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = rstd * (g - c1 - h * c2)
    d = depth(n) + 8
    e = U32 * rstd * (4 * g.abs() + 3 * c1.abs() + 6 * (h * c2).abs()
                      + d * (g.abs().mean(1, keepdim=True)
                             + h.abs() * (g * h).abs().mean(1, keepdim=True)))
    deep = U32 * (dy.shape[0] + 60)
    return (dx, (dy * h).sum(0), dy.sum(0)), (e, deep * (dy * h).abs().sum(0), deep * dy.abs().sum(0))


def check_backward(norm, x, dy, w, ptype=F32):
    _, mean, rstd = norm.layer_norm(x, w)
    _, codes, _ = norm.layer_norm_checkpoint(x, w)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    want, bound = backward64(dy, h, rstd, w)
    got = norm.layer_norm_backward(dy, x, mean, rstd, w, param_dtype=ptype)
    # From x, h itself takes two roundings; they scale every term of dx by at most that.
    for i, name in enumerate(("dx", "dw", "db")):
        t = dy.dtype if i == 0 else ptype
        assert got[i].dtype == t
        within(got[i], want[i], bound[i] + rounding(want[i], t), f"{name} from x")
    h = codes.view(torch.float8_e4m3fn).double() / norm.checkpoint_scale(x.shape[1])
    want, bound = backward64(dy, h, rstd, w)
    got = norm.layer_norm_checkpoint_backward(dy, codes, rstd, w, param_dtype=ptype)
    for i, name in enumerate(("dx", "dw", "db")):
        t = dy.dtype if i == 0 else ptype
        within(got[i], want[i], bound[i] + rounding(want[i], t), f"{name} from codes")
    alone = norm.layer_norm_checkpoint_backward(dy, codes, rstd, w, param_grads=False)
    assert torch.equal(alone[0], got[0]) and alone[1] is None and alone[2] is None


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("hidden", WIDTHS)
def test_backward(norm, hidden, dtype, ptype):
    rows = 6 if hidden > 16 else 41
    announce(f"backward {rows}x{hidden} {dtype} {ptype}")
    x, dy = rows_of(rows, hidden, dtype, 51, 2.0, 0.5), rows_of(rows, hidden, dtype, 52, 0.1)
    check_backward(norm, x, dy, params(hidden, ptype, 8)[0], ptype)


@pytest.mark.parametrize("rows,hidden", [(1, 2560), (9000, 40), (5000, 200), (2500, 1024),
                                         (2100, 2560), (1100, 12288), (150, 20000)])
def test_backward_many_rows(norm, rows, hidden):
    announce(f"backward {rows}x{hidden}")
    x, dy = rows_of(rows, hidden, BF, 61), rows_of(rows, hidden, BF, 62)
    check_backward(norm, x, dy, params(hidden, F32, 2)[0])


@pytest.mark.parametrize("pitch,offset", [(8, 0), (5, 0), (0, 1), (24, 8)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_backward_strides(norm, dtype, pitch, offset):
    for hidden in (72, 1001, 2568, 17000):
        announce(f"backward strides {hidden} {dtype} pitch {pitch} offset {offset}")
        x = rows_of(7, hidden, dtype, 71, pitch=pitch, offset=offset)
        dy = rows_of(7, hidden, dtype, 72, pitch=pitch + 8)
        check_backward(norm, x, dy, params(hidden, F32, 2)[0])


def test_backward_without_weight_and_in_place(norm):
    for hidden in (40, 2560, 20000):
        announce(f"backward in place {hidden}")
        x, dy = rows_of(600, hidden, BF, 81), rows_of(600, hidden, BF, 82)
        check_backward(norm, x, dy, None)
        _, mean, rstd = norm.layer_norm(x)
        want = norm.layer_norm_backward(dy, x, mean, rstd)
        got = norm.layer_norm_backward(dy, x, mean, rstd, dx=dy)
        assert got[0] is dy and all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_against_differences(norm):
    """Directional differences of sum(y * dy) in 64 bits, around the kernel's
    inputs: a central difference of step t is off by O(t^2)."""
    announce("differences")
    rows, hidden, eps, t = 4, 96, 1e-5, 1e-4
    x, dy = rows_of(rows, hidden, F32, 91), rows_of(rows, hidden, F32, 92)
    w, b = params(hidden, F32, 12)
    _, mean, rstd = norm.layer_norm(x, w, b, eps)
    dx, dw, db = norm.layer_norm_backward(dy, x, mean, rstd, w)
    value = lambda x, w, b: (Forward64(x, w, b, eps).y * dy.double()).sum()  # noqa: E731
    for which, grad in enumerate((dx, dw, db)):
        at = [x.double(), w.double(), b.double()]
        step = torch.zeros_like(at[which]).normal_(generator=gen(93 + which))
        hi, lo = list(at), list(at)
        hi[which], lo[which] = at[which] + t * step, at[which] - t * step
        slope = (value(*hi) - value(*lo)) / (2 * t)
        scale = (grad.double() * step).abs().sum()
        assert abs(float((grad.double() * step).sum() - slope)) <= float(scale) * 1e-5


# -------------------------------------------------------------- empty sums --

def test_no_rows(norm):
    announce("no rows")
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    w, b = params(64, F32, 1)
    y, mean, rstd = norm.layer_norm(x, w, b)
    y, codes, rstd = norm.layer_norm_checkpoint(x, w, b)
    assert y.shape == codes.shape == (0, 64) and mean.numel() == rstd.numel() == 0
    for out in (norm.layer_norm_backward(x, x, mean, rstd, w),
                norm.layer_norm_checkpoint_backward(x, codes, rstd, w)):
        assert out[0].shape == (0, 64)
        assert torch.equal(out[1], torch.zeros(64, device="cuda"))
        assert torch.equal(out[2], torch.zeros(64, device="cuda"))
    dz = torch.empty(0, 24, device="cuda", dtype=BF)
    dW, db = norm.checkpoint_weight_grad(dz, codes, w, b)
    assert dW.shape == (24, 64) and not dW.any() and not db.any()
    acc = torch.ones(24, 64, device="cuda")
    norm.checkpoint_weight_grad(dz, codes, w, b, out=acc, accumulate=True)
    assert torch.equal(acc, torch.ones_like(acc))


# ------------------------------------------------------------- weight grad --

def check_weight_grad(norm, dy, codes, w, b, dtype=None, accumulate=False):
    rows, hidden = codes.shape
    h = codes.view(torch.float8_e4m3fn).double() / norm.checkpoint_scale(hidden)
    one = torch.ones(hidden, device="cuda", dtype=torch.float64)
    wd = one if w is None else w.double()
    bd = 0 * one if b is None else b.double()
    d = dy.double()
    db = d.sum(0)
    want = (d.t() @ h) * wd + db[:, None] * bd
    size = (d.t().abs() @ h.abs()) * wd.abs() + d.abs().sum(0)[:, None] * bd.abs()
    out = None
    dtype = dy.dtype if dtype is None else dtype
    if accumulate:
        out = torch.empty(want.shape, device="cuda").normal_(generator=gen(5))
        want = want + out.double()
        size = size + out.double().abs()
    got, got_db = norm.checkpoint_weight_grad(dy, codes, w, b, out=out, dtype=dtype,
                                              accumulate=accumulate)
    assert got.dtype == dtype
    deep = U32 * (rows + 24)
    within(got_db, db, deep * d.abs().sum(0) + 1e-30, "db")
    within(got, want, deep * size + rounding(want, dtype), "dW")
    return got


def codes_of(norm, rows, hidden, seed, ptype=F32):
    w, b = params(hidden, ptype, seed)
    x = rows_of(rows, hidden, BF if ptype == F32 else ptype, seed)
    _, codes, _ = norm.layer_norm_checkpoint(x, w, b)
    return codes, w, b


# Single elements, both sides of a tile's depth (64) and width (128, 256),
# ragged everything, split sums, and enough tiles for the larger ones.
SHAPES = [(1, 1, 1), (1, 8, 16), (2, 3, 5), (63, 24, 48), (64, 128, 128), (65, 130, 257),
          (127, 120, 144), (200, 256, 512), (1000, 1030, 1111), (513, 7, 2000), (4096, 136, 144),
          (5000, 40, 33), (300, 4096, 2560), (129, 4104, 2576), (77, 4099, 2571),
          (64, 12288, 1024), (1100, 3584, 3600)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows,features,hidden", SHAPES)
def test_weight_grad(norm, rows, features, hidden, dtype):
    announce(f"weight grad {rows} {features} {hidden} {dtype}")
    codes, w, b = codes_of(norm, rows, hidden, 101, dtype)
    dy = rows_of(rows, features, dtype, 102, 0.1)
    check_weight_grad(norm, dy, codes, w, b)
    check_weight_grad(norm, dy, codes, w.float(), None, dtype=F32)
    check_weight_grad(norm, dy, codes, None, b.float(), dtype=F32, accumulate=True)


@pytest.mark.parametrize("rows,features,hidden", [(16999, 411, 5478), (10889, 5475, 809),
                                                  (16992, 2944, 1824), (6000, 4160, 5664)])
def test_weight_grad_with_tiles_cut_unevenly(norm, rows, features, hidden):
    """Long sums over tiles that do not divide among the CUs: 44, 88, 96 and
    256 + 135 tiles, whose steps are shared out across their borders."""
    announce(f"weight grad, tiles cut unevenly {rows} {features} {hidden}")
    codes, w, b = codes_of(norm, rows, hidden, 103)
    dy = rows_of(rows, features, BF, 104, 0.1)
    got = check_weight_grad(norm, dy, codes, w, b)
    assert torch.equal(got, norm.checkpoint_weight_grad(dy, codes, w, b)[0])


@pytest.mark.parametrize("pitch,offset", [(8, 0), (5, 0), (0, 1), (16, 8)])
def test_weight_grad_strides(norm, pitch, offset):
    for rows, features, hidden in ((130, 136, 144), (70, 4096, 2560)):
        announce(f"weight grad strides {rows} {features} {hidden} pitch {pitch} offset {offset}")
        codes, w, b = codes_of(norm, rows, hidden, 111)
        dy = rows_of(rows, features, BF, 112, pitch=pitch, offset=offset)
        check_weight_grad(norm, dy, codes, w, b)
        flat = torch.empty(codes.numel() + 4, device="cuda", dtype=torch.uint8)
        shifted = flat[3:3 + codes.numel()].view(codes.shape).copy_(codes)
        check_weight_grad(norm, dy, shifted, w, b)


def test_weight_grad_holds_every_code(norm):
    """All finite E4M3 values against one-hot gradients: exact."""
    announce("weight grad, every code")
    codes = torch.arange(256, device="cuda", dtype=torch.uint8).repeat(256, 1)
    codes[(codes & 0x7F) == 0x7F] = 0
    for dtype in (BF, F16):
        dy = torch.eye(256, device="cuda", dtype=dtype) * 0.5
        got, db = norm.checkpoint_weight_grad(dy, codes, dtype=F32)
        want = codes.view(torch.float8_e4m3fn).float() * 0.5 / norm.checkpoint_scale(256)
        assert torch.equal(got, want) and torch.equal(db, torch.full_like(db, 0.5))


@pytest.mark.parametrize("dtype", [BF, F16])
def test_weight_grad_of_subnormal_gradients(norm, dtype):
    """The smallest values of the type are not flushed to zero."""
    announce(f"weight grad, subnormal {dtype}")
    codes = torch.full((256, 16), 0x38, device="cuda", dtype=torch.uint8)          # 1.0
    dy = torch.zeros(256, 256, device="cuda", dtype=dtype)
    info = torch.finfo(dtype)
    value = info.tiny * info.eps * torch.arange(1, 257, device="cuda", dtype=torch.float64)
    dy.copy_(torch.diag(value))
    got, db = norm.checkpoint_weight_grad(dy, codes, dtype=F32)
    want = value / norm.checkpoint_scale(16)
    # bf16 subnormals are float32 subnormals: exact down to float32's own steps.
    within(got, want[:, None].expand(256, 16), torch.finfo(F32).tiny * U32 * 2, "dW")
    within(db, value, torch.finfo(F32).tiny * U32 * 2, "db")


def test_weight_grad_nan_stays_in_its_place(norm):
    announce("weight grad, NaN")
    codes, w, b = codes_of(norm, 70, 300, 121)
    dy = rows_of(70, 200, BF, 122)
    good = norm.checkpoint_weight_grad(dy, codes, w, b)[0]
    dy[69, 199] = float("nan")
    codes[3, 7] = 0x7F
    bad = norm.checkpoint_weight_grad(dy, codes, w, b)[0]
    assert bad[199].isnan().all() and bad[:, 7].isnan().all()
    keep = torch.ones_like(good, dtype=torch.bool)
    keep[199], keep[:, 7] = False, False
    assert torch.equal(bad[keep], good[keep])


# ----------------------------------------------------------- how it is run --

def all_operators(norm, x, dy, dz, w, b, stream=None):
    y, mean, rstd = norm.layer_norm(x, w, b, stream=stream)
    y2, codes, rstd2 = norm.layer_norm_checkpoint(x, w, b, stream=stream)
    return [y, mean, rstd, y2, codes, rstd2,
            *norm.layer_norm_backward(dy, x, mean, rstd, w, stream=stream),
            *norm.layer_norm_checkpoint_backward(dy, codes, rstd, w, stream=stream),
            *norm.checkpoint_weight_grad(dz, codes, w, b, stream=stream)]


def inputs(rows=700, hidden=1032, features=520):
    return (rows_of(rows, hidden, BF, 131), rows_of(rows, hidden, BF, 132),
            rows_of(rows, features, BF, 133), *params(hidden, F32, 13))


def test_results_repeat(norm):
    announce("repeat")
    args = inputs()
    first = all_operators(norm, *args)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(all_operators(norm, *args), first))


def test_other_stream(norm):
    announce("other stream")
    args = inputs()
    want = all_operators(norm, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_operators(norm, *args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_replays(norm):
    announce("graph")
    args = inputs()
    static = [t.clone() for t in args]
    all_operators(norm, *static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_operators(norm, *static)
    for turn in range(4):
        for s, t in zip(static, args):
            s.copy_(t * (1 + turn))
        want = all_operators(norm, *static)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), turn


def test_offsets_past_32_bits(norm):
    """More than 2^32 bytes of activations and 2^31 codes: the last rows."""
    announce("large")
    rows, hidden = 270000, 8192
    x = torch.empty(rows, hidden, device="cuda", dtype=BF)
    x.view(-1, 1 << 20 if x.numel() % (1 << 20) == 0 else hidden).normal_(generator=gen(141))
    w, b = params(hidden, F32, 14)
    y, codes, rstd = norm.layer_norm_checkpoint(x, w, b)
    tail = norm.layer_norm_checkpoint(x[-5:], w, b)
    for t, whole in zip(tail, (y, codes, rstd)):
        assert torch.equal(whole[-5:], t)
    dx, dw, db = norm.layer_norm_checkpoint_backward(y, codes, rstd, w, dx=y)
    want = norm.layer_norm_checkpoint_backward(tail[0], tail[1], tail[2], w)[0]
    assert torch.equal(dx[-5:], want)
    dz = torch.zeros(rows, 8, device="cuda", dtype=BF)
    dz[-3] = 1.0
    got, _ = norm.checkpoint_weight_grad(dz, codes, dtype=F32)
    row = codes[-3].view(torch.float8_e4m3fn).float() / norm.checkpoint_scale(hidden)
    assert torch.equal(got, row.expand(8, hidden))


# --------------------------------------------------------------- autograd --

def test_norm_autograd(norm):
    announce("autograd norm")
    x = rows_of(60, 200, F32, 151).view(3, 20, 200).requires_grad_()
    w, b = (p.requires_grad_() for p in params(200, F32, 15))
    dy = rows_of(60, 200, F32, 152).view(3, 20, 200)
    got = torch.autograd.grad((norm.norm(x, w, b) * dy).sum(), (x, w, b))
    ref = [t.detach().double().requires_grad_() for t in (x, w, b)]
    d = ref[0] - ref[0].mean(-1, keepdim=True)
    y = d / ((d * d).mean(-1, keepdim=True) + 1e-5).sqrt() * ref[1] + ref[2]
    want = torch.autograd.grad((y * dy.double()).sum(), ref)
    for g, r in zip(got, want):
        assert g.shape == r.shape
        assert float((g.double() - r).norm() / r.norm()) <= 200 * U32
    # An expanded gradient (rows that overlap) is copied, not refused.
    assert torch.autograd.grad(norm.norm(x, w, b).sum(), b)[0].eq(60).all()
    # Without parameters, and with a bias alone.
    assert norm.norm(x).shape == x.shape
    assert torch.autograd.grad(norm.norm(x, None, b).sum(), b)[0].eq(60).all()


@pytest.mark.parametrize("dtype,ptype", [(BF, F32), (F16, F16)])
def test_norm_linear_autograd(norm, dtype, ptype):
    """Against the same layer in 64 bits with h replaced by its checkpoint: dW,
    dw and db then differ by roundings alone (dy = dz W is rounded to the
    activations' type by the library product: one more half step)."""
    announce(f"autograd norm_linear {dtype}")
    rows, hidden, features = 96, 160, 72
    x = rows_of(rows, hidden, dtype, 161).view(4, 24, hidden).requires_grad_()
    w, b = (p.requires_grad_() for p in params(hidden, ptype, 16))
    W = rows_of(features, hidden, dtype, 162, 0.05).contiguous().requires_grad_()
    c = rows_of(1, features, dtype, 163)[0].contiguous().requires_grad_()
    dz = rows_of(rows, features, dtype, 164).view(4, 24, features)
    z = norm.norm_linear(x, w, b, W, c)
    got = torch.autograd.grad(z, (x, w, b, W, c), dz)
    y, codes, rstd = norm.layer_norm_checkpoint(x.detach(), w.detach(), b.detach())
    assert torch.equal(z, torch.nn.functional.linear(y, W, c))
    h = codes.view(torch.float8_e4m3fn).double().view(rows, hidden) / norm.checkpoint_scale(hidden)
    d = dz.double().view(rows, features)
    dy = d @ W.detach().double()
    (dx, dw, db), _ = backward64(dy, h, rstd, w.detach())
    y64 = h * w.detach().double() + b.detach().double()
    want = (dx.view(x.shape), dw, db, d.t() @ y64, d.sum(0))
    for name, g, r in zip(("x", "w", "b", "W", "c"), got, want):
        assert g.shape == r.shape
        # Two roundings to the type (dy and the result), in the 2-norm.
        assert float((g.double() - r).norm() / r.norm()) <= 2 * half_step(dtype), name


def test_general_path_equals_the_usual_one(norm):
    """With a stream given, the calls take the Python path to the C ABI."""
    announce("general path")
    for args in (inputs(), inputs(33, 77, 19)):
        want = all_operators(norm, *args)
        got = all_operators(norm, *args, stream=torch.cuda.current_stream())
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_on_the_device(norm):
    announce("refusals")
    x = rows_of(4, 64, BF, 171)
    w, b = params(64, F32, 18)
    y, codes, rstd = norm.layer_norm_checkpoint(x, w, b)
    for call in (lambda: norm.layer_norm(x.double()), lambda: norm.layer_norm(x, w[:63]),
                 lambda: norm.layer_norm(x, w, b.to(BF)), lambda: norm.layer_norm(x[:, ::2]),
                 lambda: norm.layer_norm(x[:1].expand(4, 64)),
                 lambda: norm.layer_norm(x, w, b, out=y[:3]),
                 lambda: norm.layer_norm_backward(y, x, rstd[:3], rstd),
                 lambda: norm.layer_norm_checkpoint_backward(y, codes[:3], rstd),
                 lambda: norm.layer_norm_checkpoint_backward(y, codes, rstd, param_dtype=F16),
                 lambda: norm.checkpoint_weight_grad(x.float(), codes),
                 lambda: norm.checkpoint_weight_grad(x, codes, accumulate=True),
                 lambda: norm.checkpoint_weight_grad(x, codes, dtype=F16),
                 lambda: norm.checkpoint_weight_grad(x, codes, out=torch.empty(64, 63, device="cuda",
                                                                              dtype=BF))):
        with pytest.raises((TypeError, ValueError)):
            call()
    for call in (lambda: norm.layer_norm(x, w, b, eps=-1.0),
                 lambda: norm.layer_norm(x, w, b, eps=float("nan")),
                 lambda: norm.layer_norm(x, out=x),
                 lambda: norm.layer_norm(torch.empty(4, 0, device="cuda", dtype=BF)),
                 lambda: norm.layer_norm_backward(y, x, rstd, rstd, dx=x)):
        with pytest.raises(norm.TacoError):
            call()


def test_example_trains_like_the_usual_layers(norm):
    announce("example")
    from gradients_taco_compress_amd import checkpointed_mlp as mlp
    plain, _ = mlp.train(512, 256, 12, False)
    ours, _ = mlp.train(512, 256, 12, True)
    assert ours[-1] < 0.9 * ours[0] and plain[-1] < 0.9 * plain[0]
    assert abs(ours[-1] - plain[-1]) <= 0.02 * plain[-1]
    p = mlp.parameters(256, 1024, 0)
    x = torch.randn(512, 256, device="cuda").to(BF).requires_grad_()
    # One byte an element and four a row, in the allocator's 512-byte steps.
    assert mlp.kept_bytes(x, p, True) <= 512 * 256 + 4 * 512 + 1024
    assert mlp.kept_bytes(x, p, False) >= 4 * 512 * 256


def test_norm_linear_keeps_one_byte_per_element(norm):
    announce("memory")
    x = torch.randn(4096, 2048, device="cuda", dtype=BF).requires_grad_()
    w, b = params(2048, F32, 17)
    W = torch.randn(8, 2048, device="cuda", dtype=BF).requires_grad_()
    norm.norm_linear(x, w, b, W).sum().backward()
    before = torch.cuda.memory_allocated()
    z = norm.norm_linear(x, w, b, W)
    kept = torch.cuda.memory_allocated() - before - z.numel() * 2
    assert kept <= x.numel() + 4 * 4096 + 4096
