"""Which tiles and cuts libtaco_gated takes for a size, for tests that have to reach
each of them: the rules of taco_gated_product.hpp and taco_gated_few.hpp again, with the
costs read out of those files, so that sizes which no longer reach a plan are noticed
when the costs change.  tests/test_gated_plans_host.py compares the workspaces that
follow from these plans with the library's."""
from __future__ import annotations

import os
import re
from collections import namedtuple

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gradients_taco_compress_amd", "csrc")

Cost = namedtuple("Cost", "places fixed step alone part")
#: tiles of `size`; `whole` of them in one piece, `split` in `parts` parts of `share`
#: K-tiles of the `depth` of each.
Plan = namedtuple("Plan", "size us tiles whole split parts share depth slab_bytes")


def up(n, d):
    return -(-n // d)


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _read():
    text = _source("taco_gated_product.hpp")
    costs = {}
    for name in ("Large", "Small", "Deep"):
        values = re.search(rf"constexpr Cost k{name}Cost = \{{([^}}]*)\}};", text).group(1).split(",")
        costs[name.lower()] = Cost(int(values[0]), *map(float, values[1:]))
    shapes = {n.lower(): (int(bm), int(ring)) for n, bm, ring in
              re.findall(r"using (Large|Small|Deep) = Shape<(\d+), \2, \d, \d, (\d)>;", text)}
    join = float(re.search(r"constexpr double kJoinUs = ([\d.]+);", text).group(1))
    splits = tuple(map(int, re.search(r"for \(int64_t split : \{([\d, ]+)\}\)", text).group(1).split(",")))
    return costs, shapes, join, splits


COSTS, SHAPES, JOIN_US, SPLITS = _read()


def _groups_us(c, groups, steps):
    left = groups % c.places
    more = max(2.0 * left / c.places - 1.0, 0.0)
    step = c.alone + (c.step - c.alone) * more
    return groups // c.places * (c.fixed + steps * c.step) + (c.fixed + steps * step if left else 0.0)


def plan_of(size, kind, m, n, k, bytes_each=2, cost=None):
    """kind: "forward", "input" or "weight"; m, n, k: rows, columns and summed length."""
    edge, ring = SHAPES[size]
    c = cost or COSTS[size]
    depth = up(k, 128 // bytes_each) * (2 if kind == "input" else 1)
    tiles = up(m, edge) * (2 if kind == "weight" else 1) * up(n, edge // 2 if kind == "forward" else edge)
    left = tiles % c.places

    def rounds(groups, steps):
        return _groups_us(c, groups, up(steps, ring) * ring)
    best = Plan(size, rounds(tiles, depth), tiles, tiles, 0, 1, depth, depth, 0)
    for split in SPLITS:
        if left == 0 or split * 4 > depth:
            break
        share = up(depth, split)
        parts = up(depth, share)
        us = rounds(tiles - left, depth) + rounds(left * parts, share) + left * parts * c.part + JOIN_US
        if us < best.us:
            best = Plan(size, us, tiles, tiles - left, left, parts, share, depth,
                        left * parts * edge * edge * 4)
    return best


def product(kind, m, n, k, bytes_each=2):
    large, small, deep = (plan_of(s, kind, m, n, k, bytes_each) for s in ("large", "small", "deep"))
    other = large if large.us <= small.us else small
    return deep if deep.us <= other.us else other


def few_takes(rows, features, hidden, bytes_each=2, copies=0):
    if rows <= 16:
        return True
    if rows > 64:
        return False
    weights = 2.0 * features * hidden * bytes_each / 5.0e6
    cu = (up(up(features, 16), 256) * (32.0 + 0.5 * (rows + (32 if rows <= 32 else 64)))
          * hidden * bytes_each / (25.0e3 if bytes_each == 1 else 34.0e3))
    p = product("forward", rows, features, hidden, bytes_each)
    join = JOIN_US + 0.015 * p.split * p.parts if p.split else 0.0
    tiles = max(p.us, 4.0 + weights + 0.8 * join) + (4.0 if bytes_each == 1 else 0.0)
    tiles += 3.0 + copies / 2.0e6 if copies else 0.0
    return 3.0 + max(cu, weights) < tiles


def forward(rows, hidden, features, bytes_each=2, copies=0):
    """The plan of a forward pass, or None where it goes without tiles."""
    if few_takes(rows, features, hidden, bytes_each, copies):
        return None
    return product("forward", rows, features, hidden, bytes_each)


def backward(rows, hidden, features):
    """(together, plan of dX, plan of the weights' gradients) of a pass that wants both."""
    x, w = product("input", rows, hidden, features), product("weight", features, hidden, rows)
    if "large" in (x.size, w.size):
        return False, x, w
    half = COSTS["small"]._replace(places=COSTS["small"].places // 2)
    return (True, plan_of("small", "input", rows, hidden, features, cost=half),
            plan_of("small", "weight", features, hidden, rows, cost=half))


# Sizes (rows, hidden, features) that reach each plan: tiles, whether some are whole,
# and whether some are split.  All edges are ragged; widths that are no multiple of 8
# go through copies of the operands.
FORWARD = {
    (71, 40, 34): ("small", True, False),
    (65, 944, 37): ("small", False, True),
    (276, 6365, 10881): ("small", True, True),
    (1292, 925, 36): ("deep", True, False),
    (3793, 14112, 37): ("deep", False, True),
    (388, 40, 8298): ("large", True, False),
    (676, 652, 11090): ("large", True, True),
    (138, 16112, 4945): ("large", False, True),
}
FORWARD_CODES = {
    (73, 32, 34): ("small", True, False),
    (67, 2176, 33): ("small", False, True),
    (880, 3840, 10105): ("small", True, True),
    (1059, 1824, 33): ("deep", True, False),
    (3462, 14304, 66): ("deep", False, True),
    (299, 32, 11142): ("large", True, False),
    (6052, 1440, 1401): ("large", True, True),
}
# dX alone, and the weights' gradients alone.
INPUT = {
    (66, 36, 35): ("small", True, False),
    (79, 32, 534): ("small", False, True),
    (878, 19593, 905): ("small", True, True),
    (3631, 43, 469): ("deep", True, False),
    (3790, 42, 6992): ("deep", False, True),
    (5174, 1575, 33): ("large", True, False),
    (6962, 130, 11190): ("large", False, True),
    (1240, 13216, 333): ("large", True, True),
}
WEIGHT = {
    (75, 32, 38): ("small", True, False),
    (976, 33, 34): ("small", False, True),
    (3531, 263, 10996): ("small", True, True),
    (930, 34, 608): ("deep", True, False),
    (6994, 38, 3721): ("deep", False, True),
    (71, 17531, 167): ("large", True, False),
    (724, 1195, 6619): ("large", True, True),
}
