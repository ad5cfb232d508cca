"""Which plans the sizes of the GPU tests reach, without a GPU: the rules as
gated_plans.py has them give the library's own workspaces, and each plan has a size."""
import random

import pytest

import gated_plans as plans

torch = pytest.importorskip("torch")
gated = pytest.importorskip("gradients_taco_compress_amd.gated")

A = 1 << 24          # fake, aligned device addresses (the workspaces' sizes look at nothing else)
TABLES = {"forward": (plans.FORWARD, plans.forward),
          "codes": (plans.FORWARD_CODES, lambda *s: plans.forward(*s, bytes_each=1)),
          "input": (plans.INPUT, lambda t, h, f: plans.product("input", t, h, f)),
          "weight": (plans.WEIGHT, lambda t, h, f: plans.product("weight", f, h, t))}


@pytest.mark.parametrize("kind", TABLES)
def test_sizes_reach_the_plans_that_they_are_listed_for(kind):
    table, rule = TABLES[kind]
    for size, (tiles, whole, split) in table.items():
        p = rule(*size)
        assert p is not None and (p.size, p.whole > 0, p.split > 0) == (tiles, whole, split), (size, p)
    assert {t[0] for t in table.values()} == {"small", "deep", "large"}
    assert {(t[0], t[2]) for t in table.values()} == {(s, b) for s in ("small", "deep", "large")
                                                      for b in (False, True)}


def test_a_part_of_dx_runs_from_the_first_sum_into_the_second():
    """Large tiles, split: parts within dG Wg, one across, and parts within dU Wu."""
    p = plans.product("input", 6962, 130, 11190)
    middle = p.depth // 2
    assert p.size == "large" and p.split
    across = [i for i in range(p.parts) if i * p.share < middle < (i + 1) * p.share]
    assert across and 0 < across[0] < p.parts - 1


def copied(rows, width):
    return rows * plans.up(width * 2, 16) * 16 if width % 8 else 0


def forward_bytes(rows, hidden, features):
    copies = copied(rows, hidden) + 2 * copied(features, hidden)
    p = plans.forward(rows, hidden, features, copies=copies)
    return 0 if p is None else p.slab_bytes + copies


def codes_bytes(rows, hidden, features):
    p = plans.forward(rows, hidden, features, bytes_each=1)
    tiles = plans.up(hidden, 128) * 256 * (plans.up(rows, 64) + 2 * plans.up(features, 64))
    return 0 if p is None else p.slab_bytes + tiles


def backward_bytes(rows, hidden, features, dx, dw):
    d = 2 * rows * plans.up(features, 8) * 16
    if dx and dw:
        together, x, w = plans.backward(rows, hidden, features)
        slabs = x.slab_bytes + w.slab_bytes if together else max(x.slab_bytes, w.slab_bytes)
    else:
        slabs = (plans.product("input", rows, hidden, features) if dx
                 else plans.product("weight", features, hidden, rows)).slab_bytes
    return d + slabs + (2 * copied(features, hidden) if dx else 0) + (copied(rows, hidden) if dw else 0)


def test_the_rules_give_the_librarys_workspaces():
    rng = random.Random(3)
    sizes = [s for table, _ in TABLES.values() for s in table]
    sizes += [tuple(int(2 ** rng.uniform(0, most)) for most in (15, 14, 14)) for _ in range(1500)]
    split = 0
    for rows, hidden, features in sizes:
        size = rows, hidden, features
        weights = (A, hidden, A, hidden)
        assert gated.taco_gated_forward_workspace(A, hidden, *weights, *size) == forward_bytes(*size), size
        for dx, dw in ((1, 1), (1, 0), (0, 1)):
            assert (gated.taco_gated_backward_workspace(A, hidden, *weights, *size, dx, dw)
                    == backward_bytes(*size, dx, dw)), (size, dx, dw)
        split += plans.product("input", rows, hidden, features).split > 0
        coded = rows, plans.up(hidden, 32) * 32, features
        assert gated.taco_gated_forward_mx_workspace(*coded) == codes_bytes(*coded), coded
    assert split > 300
