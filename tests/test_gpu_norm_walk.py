"""The kernels of layer norm where a work-group takes several rows: every forward
kernel over three turns at least.  What lies between rows is NaN.
"""
from __future__ import annotations

import pytest
import torch

from test_gpu_norm import BF, F16, F32, announce, check_forward, norm, params, rows_of  # noqa: F401

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
@pytest.mark.parametrize("rows", [1024, 1025])
def test_forward_where_its_kernel_changes(norm, rows, hidden, dtype, ptype):  # noqa: F811
    announce(f"forward {rows}x{hidden} {dtype} {ptype}")
    w, b = params(hidden, ptype, 3)
    check_forward(norm, rows_of(rows, hidden, dtype, 11), w, b)
