"""What the exact sums of the layer norm's GPU tests can see, without a GPU."""
import pytest

torch = pytest.importorskip("torch")


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
