"""The autograd wiring of norm.rms without a GPU: the kernels' calls are replaced by
their formulas on host tensors, so that what is tested is which gradients arrive
where, and what memory they are in."""
import pytest

torch = pytest.importorskip("torch")
norm = pytest.importorskip("gradients_taco_compress_amd.norm")


def forward(x, weight=None, eps=1e-5, residual=None):
    total = x if residual is None else x + residual.reshape(x.shape)
    q = (total.square().mean(-1, keepdim=True) + eps).rsqrt()
    y = total * q * (1.0 if weight is None else weight.flatten())
    return y, None if residual is None else total, q.flatten()


def backward(dy, x, rstd, weight=None, dtotal=None, param_grads=True):
    q = rstd.view(*x.shape[:-1], 1)
    h, g = x * q, dy * (1.0 if weight is None else weight.flatten())
    dx = q * (g - h * (g * h).mean(-1, keepdim=True))
    dx = dx if dtotal is None else dx + dtotal
    return dx, (dy * h).flatten(0, -2).sum(0) if param_grads else None


@pytest.fixture
def rms(monkeypatch):
    monkeypatch.setattr(norm, "rms_norm", forward)
    monkeypatch.setattr(norm, "rms_norm_backward", backward)
    monkeypatch.setattr(norm, "_even", lambda t: t)
    return norm.rms


def leaves(*shapes):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(s, dtype=torch.float64, generator=g).requires_grad_() for s in shapes]


class Untouched(torch.autograd.Function):
    """Passes a value on and no gradient back."""

    @staticmethod
    def forward(ctx, y):
        return y.clone()

    @staticmethod
    def backward(ctx, dy):
        return None


def test_outputs_without_gradients(rms):
    x, r, w = leaves((3, 8), (3, 8), (8,))
    y, total = rms(x, w, residual=r)
    (Untouched.apply(y).sum() + (x * 2).sum()).backward()       # neither y nor the sum has one
    assert torch.equal(x.grad, torch.full_like(x, 2.0)) and r.grad is None and w.grad is None
    y, total = rms(x, w, residual=r)
    x.grad = None
    (Untouched.apply(y).sum() + (total * 3).sum()).backward()   # the sum alone
    assert torch.equal(x.grad, torch.full_like(x, 3.0)) and torch.equal(r.grad, x.grad)
    assert w.grad is None or not bool(w.grad.any())


@pytest.mark.parametrize("shape", [(3, 8), (1, 3, 8)])
def test_gradients_have_memory_of_their_own(rms, shape):
    """Where y is not used the sum's gradient is that of x and of the residual: three
    gradients that a caller may each add to."""
    x, r, w = leaves((3, 8), shape, (8,))
    one = torch.ones(3, 8, dtype=torch.float64)
    rms(x, w, residual=r)[1].backward(one)
    places = [t.untyped_storage().data_ptr() for t in (x.grad, r.grad, one)]
    assert len(set(places)) == 3
    rms(x, w, residual=r)[1].backward(one)                      # adds to both in place
    assert bool((one == 1).all()) and bool((x.grad == 2).all()) and bool((r.grad == 2).all())
    assert r.grad.shape == r.shape
    # through another addition, whose other side receives the same gradient
    x, r, w, z = leaves((3, 8), shape, (8,), (3, 8))
    (rms(x, w, residual=r)[1] + z).backward(one)
    for t in (x, r, z):
        t.grad.add_(1)
    assert all(bool((t.grad == 2).all()) for t in (x, r, z)) and bool((one == 1).all())
    # the residual alone
    x, r, w = leaves((3, 8), shape, (8,))
    rms(x.detach(), w.detach(), residual=r)[1].backward(one)
    assert r.grad.untyped_storage().data_ptr() != one.untyped_storage().data_ptr()
    # both outputs
    x, r, w = leaves((3, 8), shape, (8,))
    torch.autograd.backward(rms(x, w, residual=r), (one, one))
    r.grad.zero_()
    assert x.grad.untyped_storage().data_ptr() != r.grad.untyped_storage().data_ptr()
    assert bool(x.grad.any())
