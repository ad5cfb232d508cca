"""Layer norm without a GPU: what its C ABI takes for an overlap, and what the exact
sums of its GPU tests can see."""
import pytest

torch = pytest.importorskip("torch")

ALIAS, PARAM = 6, 4
A = 1 << 24          # a fake, aligned device address


def test_exact_sums_see_every_row():
    """The planted mistake is in the oracle: with any one row left out of it, or
    taken twice, sums of these whole numbers differ wherever one looks."""
    from test_gpu_norm_walk import CODE_OF
    rows, features, hidden = 4099, 24, 40
    g = torch.Generator().manual_seed(1)
    dy = torch.tensor([-2.0, -1.0, 1.0, 2.0])[torch.randint(0, 4, (rows, features), generator=g)]
    v = torch.tensor(list(CODE_OF))[torch.randint(0, len(CODE_OF), (rows, hidden), generator=g)]
    dy, v = dy.double(), v.double()
    full, db = dy.t() @ v, dy.sum(0)
    for at in (0, 31, 32, 2048, rows - 1):
        once = torch.ones(rows, 1, dtype=torch.float64)
        for times in (0.0, 2.0):
            once[at] = times
            assert bool(((dy * once).t() @ v != full).all())
            assert bool(((dy * once).sum(0) != db).all())


def side_by_side(dy, x, dx, ld=256, ldx=None, lddx=None, rows=5, hidden=64):
    """Status of a float32 backward call whose activations start at these columns
    of one buffer.  Its workspace is a byte short, which is found after overlaps
    and before anything is launched."""
    norm = pytest.importorskip("gradients_taco_compress_amd.norm")
    need = norm.taco_norm_backward_workspace(rows, hidden)
    return norm.taco_norm_backward(
        A + 4 * dy, ld, A + 4 * x, ldx or ld, 3 * A, 4 * A, 0, rows, hidden, 2, 2, A + 4 * dx,
        lddx or ld, 7 * A, 8 * A, 9 * A, need - 1, 0)


def test_column_slices_of_one_tensor_do_not_overlap():
    assert side_by_side(0, 64, 128) == PARAM
    assert side_by_side(128, 64, 0) == PARAM                 # before the inputs
    assert side_by_side(0, 64, 192) == PARAM                 # up to the next row
    assert side_by_side(0, 64, 2 * 256 + 128) == PARAM       # two rows further down
    assert side_by_side(2 * 256, 2 * 256 + 64, 128) == PARAM
    assert side_by_side(0, 64, 5 * 256) == PARAM             # behind all rows
    assert side_by_side(0, 64, 64 + 4 * 256 + 64) == PARAM


def test_rows_that_share_elements_overlap():
    for dx in (1, 63, 65, 127, 64, 193, 255, 256, 4 * 256 + 1):
        assert side_by_side(0, 64, dx) == ALIAS, dx
    assert side_by_side(256, 256 + 64, 193) == ALIAS         # runs into the inputs' first row
    assert side_by_side(0, 0, 0, ld=64) == ALIAS             # dx is dy, and x too
    assert side_by_side(0, 1 << 20, 0) == PARAM              # dx is dy


def test_rows_of_different_pitches_overlap_where_their_extents_do():
    assert side_by_side(0, 1 << 20, 128, lddx=512) == ALIAS
    assert side_by_side(0, 64, 128, ldx=512) == ALIAS        # x's rows pass under dx's
    assert side_by_side(0, 1 << 20, 5 * 256, lddx=512) == PARAM


def test_every_overlap_of_short_rows_is_found():
    """All placements of three rows against three, by elements."""
    rows, pitch = 3, 8
    for width in (1, 3, 4, 7, 8):
        for at in range(-3 * pitch, 3 * pitch + 1):
            held = {r * pitch + c for r in range(rows) for c in range(width)}
            dx = {at + r * pitch + c for r in range(rows) for c in range(width)}
            want = ALIAS if held & dx and at != 0 else PARAM
            assert side_by_side(0, 1 << 20, at, ld=pitch, rows=rows, hidden=width) == want, (width, at)
