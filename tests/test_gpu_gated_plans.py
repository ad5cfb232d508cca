"""Every plan of the gated block's products on the GPU, with sums that are exact.

The sizes are gated_plans.py's (which plan each reaches is tested without a GPU):
256x256 and 128x128 tiles in two K-tiles of LDS and 128x128 ones in four, in one
piece and in parts, all edges ragged.  Operands are whole numbers times powers of two, so
that every order of summing gives the same float32 value: G, U and the gradients have to
be equal to the 64-bit ones rounded once, and A is off by the activation's float32
error alone (gated_reference.py).  Around operands whose rows are a multiple of 16
bytes lie NaN.  Every case prints its name before it touches the GPU.
"""
from __future__ import annotations

import math

import pytest
import torch

import gated_plans as plans
from gated_reference import ACTIVATIONS, BF, F16, U32, Activation, rounding, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gated():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gradients_taco_compress_amd.gated as gated
    return gated


def announce(msg):
    print(f"[case] {msg}", flush=True)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def whole(rows, width, seed, most=1):
    return torch.randint(-most, most + 1, (rows, width), generator=gen(seed), device="cuda").float()


def powers(n, low, high, seed):
    return torch.exp2(torch.randint(low, high + 1, (n,), generator=gen(seed), device="cuda").float())


def surrounded(t, dtype):
    """t in rows 8 elements further apart, NaN between them (contiguous where its
    rows are copied anyway)."""
    if t.shape[1] % 8:
        return t.to(dtype)
    full = torch.full((t.shape[0], t.shape[1] + 8), float("nan"), device="cuda", dtype=dtype)
    full[:, :-8] = t
    return full[:, :-8]


def check_activation(a, g, u, kind):
    """A against act(g) u, g and u (float64) being what the kernel holds exactly."""
    act = Activation(g, kind)
    value, e_value = act.act, act.e_act
    if kind == "gelu":
        # The normal distribution's function by erfc: torch's ndtr is 1 + erf there, which
        # has no digits left where it is below 2^-53 (g < -8), and these gates go to -50.
        p = 0.5 * torch.erfc(g * -0.5 ** 0.5)
        phi = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        value = g * p
        e_value = g.abs() * (g.abs() * phi * 4 + 64 * p) * U32 + 4 * U32 * value.abs() + 1e-37
    # act = g share, and share is a float32 number: 0 where it is below the smallest, 2^-126
    # (silu of g < -87.3), so that act loses up to |g| 2^-126 there.
    e_value = e_value + g.abs() * 2.0 ** -126
    want = value * u
    error = e_value * u.abs() + 4 * U32 * want.abs() + 1e-37
    within(a, want, error + rounding(want.abs() + error, a.dtype), "a")


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows,hidden,features", plans.FORWARD)
def test_forward(gated, rows, hidden, features, dtype):
    kind = ACTIVATIONS[(rows + (dtype is F16)) % 3]
    announce(f"plans forward {rows} x {features}x{hidden} {dtype} {kind}")
    # sums below 2^15 in steps of 1/8: exact, and A stays within float16
    x, wg, wu = (whole(n, hidden, i) for i, n in enumerate((rows, features, features)))
    x = x / 8
    a, gate, up = gated.gated_forward(*(surrounded(t, dtype) for t in (x, wg, wu)), kind, save=True)
    g, u = (x.double() @ w.double().t().contiguous() for w in (wg, wu))
    assert torch.equal(gate, g.to(dtype)) and torch.equal(up, u.to(dtype))
    check_activation(a, g, u, kind)
    again = gated.gated_forward(*(surrounded(t, dtype) for t in (x, wg, wu)), kind)
    assert torch.equal(a, again)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows,hidden,features", plans.FORWARD_CODES)
def test_forward_from_codes(gated, rows, hidden, features, dtype):
    """Rows, features and blocks along the summed index each have a scale of their own
    (the blocks' reciprocal, so that sums stay exact): a scale of another place shows."""
    kind = ACTIVATIONS[(rows + (dtype is F16)) % 3]
    announce(f"plans codes {rows} x {features}x{hidden} {dtype} {kind}")
    x, wg, wu = (whole(n, hidden, i) for i, n in enumerate((rows, features, features)))
    x[:, ::32] = 1.0                                                # no block of zeros
    wg[:, ::32], wu[:, 1::32] = -1.0, 1.0
    block = powers(hidden // 32, -6, 6, 4).repeat_interleave(32)
    x = x * powers(rows, -8, -3, 5)[:, None] * block
    wg, wu = (w * powers(features, -3, 1, 6 + i)[:, None] / block for i, w in enumerate((wg, wu)))
    pairs = [gated.mx_encode(t) for t in (x, wg, wu)]
    assert min(scales.unique().numel() for _, scales in pairs) >= 5      # (rows have scales of their own)
    a = gated.gated_forward_mx(*pairs, kind, dtype=dtype)
    g, u = (x.double() @ w.double().t().contiguous() for w in (wg, wu))
    check_activation(a, g, u, kind)


def backward_operands(rows, hidden, features, dtype):
    """silu(64) = 64 and its slope is 1 in float32: dG = dA U and dU = 64 dA are whole
    numbers, and so are all sums."""
    da, up = whole(rows, features, 1), whole(rows, features, 2)
    x, wg, wu = (whole(n, hidden, 3 + i) for i, n in enumerate((rows, features, features)))
    gate = torch.full((rows, features), 64.0, device="cuda")
    args = [surrounded(t, dtype) for t in (da, x, gate, up, wg, wu)]
    return args, da * up, da * 64, x, wg, wu


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows,hidden,features", plans.INPUT)
def test_input_gradient(gated, rows, hidden, features, dtype):
    announce(f"plans dX {rows} x {features}x{hidden} {dtype}")
    args, dgate, dup, x, wg, wu = backward_operands(rows, hidden, features, dtype)
    dx, none, also = gated.gated_backward(*args, weight_grads=False)
    assert none is None and also is None
    assert torch.equal(dx, (dgate.double() @ wg.double() + dup.double() @ wu.double()).to(dtype))
    assert torch.equal(dx, gated.gated_backward(*args)[0])


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows,hidden,features", plans.WEIGHT)
def test_weight_gradients(gated, rows, hidden, features, dtype):
    announce(f"plans dWg, dWu {rows} x {features}x{hidden} {dtype}")
    args, dgate, dup, x, wg, wu = backward_operands(rows, hidden, features, dtype)
    none, dg, du = gated.gated_backward(*args, input_grad=False)
    assert none is None
    for got, d in ((dg, dgate), (du, dup)):
        assert torch.equal(got, (d.t().contiguous().double() @ x.double()).to(dtype))
    _, dg2, du2 = gated.gated_backward(*args)
    assert torch.equal(dg, dg2) and torch.equal(du, du2)
