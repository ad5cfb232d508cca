"""The kernels of layer norm where a work-group takes several rows or pieces:
every forward kernel over at least three turns, the backward kernels' walk with
its two rows in flight, and the cut points of the sums over rows.

Where a sum over rows is checked, its terms are small whole numbers and powers
of two, so that float32 holds every partial sum exactly and a lost, doubled or
misplaced row cannot hide in a tolerance.  What lies between rows is NaN.
"""
from __future__ import annotations

import pytest
import torch

from test_gpu_norm import (BF, F16, F32, announce, backward64, check_forward, gen, norm,  # noqa: F401
                           params, rounding, rows_of, within)

pytestmark = pytest.mark.gpu

TYPES = [(BF, F32), (BF, BF), (F16, F32), (F16, F16), (F32, F32)]

# --------------------------------------------------------------- forward --

# (rows that are in flight at once, widths): both sides of each limit of the
# kernels for many rows, in whole chunks and ragged.
FORWARD = [(32768, (8, 127, 128)), (16384, (129, 136, 256)), (8192, (257, 511, 512)),
           (4096, (513, 520, 1000, 1024)), (2048, (1025, 1032, 1111, 1536)),
           (2048, (1537, 1544, 2047, 2048)), (2048, (2049, 2056, 2560)),
           (2048, (2561, 2568, 3001, 3064)), (2048, (3080, 3583, 3584)),
           (2048, (3585, 3592, 4095, 4096)), (512, (4097, 4104, 6144)), (512, (6145, 8191, 8192)),
           (512, (8193, 12287, 12288)), (512, (12296, 16383, 16384)), (512, (16385, 16392))]


def nan_between(t):
    """t in a wider buffer, five columns wider, with NaN around its rows."""
    rows, hidden = t.shape
    full = torch.full((rows + 1, hidden + 5), float("nan"), device="cuda", dtype=t.dtype)
    inside = full[:rows, 1:1 + hidden]
    inside.copy_(t)
    return inside


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("flight,hidden", [(f, h) for f, widths in FORWARD for h in widths])
def test_forward_takes_several_rows(norm, flight, hidden, dtype, ptype):  # noqa: F811
    rows = 2 * flight + flight // 2 + 3
    announce(f"forward {rows}x{hidden} {dtype} {ptype}")
    x = rows_of(rows, hidden, dtype, hidden, 1.5, 0.3)
    w, b = params(hidden, ptype, 7)
    check_forward(norm, x, w, b)
    check_forward(norm, nan_between(x), w, b)             # off 16-byte boundaries


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("hidden", [520, 1111, 2560, 4096])
@pytest.mark.parametrize("rows", [512, 513, 1024, 1025])
def test_forward_where_its_kernel_changes(norm, rows, hidden, dtype, ptype):  # noqa: F811
    announce(f"forward {rows}x{hidden} {dtype} {ptype}")
    w, b = params(hidden, ptype, 3)
    check_forward(norm, rows_of(rows, hidden, dtype, 11), w, b)


# -------------------------------------------------------------- backward --

BACKWARD = [40, 77, 128, 136, 500, 512, 1001, 1024, 1111, 2048, 2571, 4096, 6001, 6144, 8191, 8192,
            12287, 12288, 16383, 16384, 16400]
LONG = [(41000, 96), (33000, 1001), (8500, 2560), (8500, 4096)]        # parts of 512 work-groups


def several_turns(hidden):
    """Rows for five and a half turns of the backward pass's work-groups."""
    per = 16 if hidden <= 128 else 4 if hidden <= 1024 else 1
    return 5 * 256 * per + 128 * per + 3


def whole(rows, hidden, dtype, seed, values):
    """[rows, hidden] of the given values, in five columns more of NaN."""
    at = torch.randint(0, len(values), (rows, hidden), device="cuda", generator=gen(seed))
    return nan_between(torch.tensor(values, device="cuda")[at].to(dtype))


# E4M3 codes of the given numbers.
CODE_OF = {0.5: 0x30, 1.0: 0x38, 2.0: 0x40, -1.0: 0xB8, -2.0: 0xC0}


def codes_and_values(rows, hidden, seed):
    value = torch.tensor(list(CODE_OF), device="cuda")
    code = torch.tensor(list(CODE_OF.values()), device="cuda", dtype=torch.uint8)
    at = torch.randint(0, len(CODE_OF), (rows, hidden), device="cuda", generator=gen(seed))
    return code[at], value[at]


@pytest.mark.parametrize("dtype,ptype", [(BF, F32), (F16, F16), (F32, F32)])
@pytest.mark.parametrize("rows,hidden", [(several_turns(h), h) for h in BACKWARD] + LONG)
def test_backward_takes_several_rows(norm, rows, hidden, dtype, ptype):  # noqa: F811
    """dx within float32's bounds, dw and db exact (float32) or rounded once."""
    announce(f"backward {rows}x{hidden} {dtype} {ptype}")
    dy = whole(rows, hidden, dtype, hidden, [-2.0, -1.0, 1.0, 2.0])
    rstd = torch.empty(rows, device="cuda").uniform_(0.5, 2.0, generator=gen(3))
    w, _ = params(hidden, ptype, 8)

    def check(got, h, r, what):
        want, bound = backward64(dy, h, r, w)
        within(got[0], want[0], bound[0] + rounding(want[0], dtype), f"dx {what}")
        assert torch.equal(got[1], want[1].to(ptype)), f"dw {what}"
        assert torch.equal(got[2], want[2].to(ptype)), f"db {what}"

    # h = (x - m) r is whole too, with r = 1.
    x = whole(rows, hidden, dtype, hidden + 1, [-3.0, -2.0, -1.0, 1.0, 2.0, 4.0])
    mean = torch.randint(-2, 3, (rows,), device="cuda", generator=gen(4)).float()
    one = torch.ones(rows, device="cuda")
    from_x = norm.layer_norm_backward(dy, x, mean, one, w)
    check(from_x, x.double() - mean.double()[:, None], one, "from x")

    codes, value = codes_and_values(rows, hidden, 5)
    from_codes = norm.layer_norm_checkpoint_backward(dy, codes, rstd, w)
    check(from_codes, value.double() / norm.checkpoint_scale(hidden), rstd, "from codes")

    # Whole chunks, where the width has them; and dx over dy.
    check(norm.layer_norm_backward(dy.contiguous(), x.contiguous(), mean, one, w),
          x.double() - mean.double()[:, None], one, "from x, contiguous")
    check(norm.layer_norm_checkpoint_backward(dy.contiguous(), codes, rstd, w),
          value.double() / norm.checkpoint_scale(hidden), rstd, "from codes, contiguous")
    before = dy.clone()
    got = norm.layer_norm_checkpoint_backward(dy, codes, rstd, w, dx=dy)
    assert got[0] is dy and all(torch.equal(a, b) for a, b in zip(got, from_codes))
    dy.copy_(before)
    got = norm.layer_norm_backward(dy, x, mean, one, w, dx=dy)
    assert got[0] is dy and all(torch.equal(a, b) for a, b in zip(got, from_x))


# ----------------------------------------------------------- weight grad --

# Rows on both sides of a tile's depth (32), of a ring of small tiles (4 of them)
# and of large ones (6), over few small tiles, many, and large ones.
DEPTHS = [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 383, 384, 385, 639]
EXACT = ([(r, 40, 48) for r in DEPTHS] + [(r, 300, 261) for r in DEPTHS]
         + [(r, 4096, 4112) for r in DEPTHS]
         # Sums split evenly, and shares cut across the tiles' borders.
         + [(4096, 136, 144), (4099, 1024, 1024), (20001, 40, 33), (32767, 64, 80), (2048, 1024, 1024),
            (9999, 513, 1000)]
         + [(16999, 411, 5478), (10889, 5475, 809), (16992, 2944, 1824), (6000, 4160, 5664)])


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows,features,hidden", EXACT)
def test_weight_grad_loses_no_row(norm, rows, features, hidden, dtype):  # noqa: F811
    announce(f"weight grad {rows} {features} {hidden} {dtype}")
    codes, value = codes_and_values(rows, hidden, 21)
    dy = whole(rows, features, dtype, 22, [-2.0, -1.0, 1.0, 2.0])
    want = (dy.double().t().contiguous() @ value.double()) / norm.checkpoint_scale(hidden)
    assert float(want.abs().max()) * norm.checkpoint_scale(hidden) < 2 ** 23
    db = dy.double().sum(0)
    # Rows on 16-byte boundaries where the width allows, with NaN behind them, and off them.
    wide = torch.full((rows, (features + 15) // 8 * 8), float("nan"), device="cuda", dtype=dtype)
    wide[:, :features] = dy
    for rows_as in (dy, wide[:, :features]):
        got, got_db = norm.checkpoint_weight_grad(rows_as, codes, dtype=F32)
        assert torch.equal(got.double(), want) and torch.equal(got_db.double(), db)
    acc = torch.full((features, hidden), 3.0, device="cuda")
    norm.checkpoint_weight_grad(wide[:, :features], codes, out=acc, accumulate=True)
    assert torch.equal(acc.double(), want + 3.0)

