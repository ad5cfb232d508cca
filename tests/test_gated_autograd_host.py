"""The autograd wiring of gated.gated without a GPU: the kernels' call is replaced by
its formula on host tensors."""
import pytest

torch = pytest.importorskip("torch")
gated = pytest.importorskip("gradients_taco_compress_amd.gated")
from torch.autograd import forward_ad  # noqa: E402


def forward(x, gate_weight, up_weight, activation="silu", save=False):
    gate, up = x @ gate_weight.t(), x @ up_weight.t()
    a = torch.nn.functional.silu(gate) * up
    return (a, gate, up) if save else a


@pytest.fixture
def block(monkeypatch):
    monkeypatch.setattr(gated, "gated_forward", lambda *args, **kw: forward(*(
        forward_ad.unpack_dual(t).primal if isinstance(t, torch.Tensor) and tangents() else t
        for t in args), **kw))                       # (the kernels take the values alone)
    monkeypatch.setattr(gated, "_even", lambda t: t)
    return gated.gated


def tangents():
    """Whether a level of forward-mode differentiation is open."""
    try:
        forward_ad.make_dual(torch.zeros(1), torch.zeros(1))
    except RuntimeError:
        return False
    return True


def operands():
    g = torch.Generator().manual_seed(1)
    return [torch.randn(s, dtype=torch.float64, generator=g) for s in ((3, 8), (5, 8), (5, 8))]


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("mode", [torch.no_grad, torch.enable_grad])
def test_tangents_are_refused(block, which, mode):
    """Forward-mode differentiation does not depend on grad mode, and the block has no
    forward-mode derivative: a tangent is refused, not dropped."""
    args = operands()
    with mode(), forward_ad.dual_level():
        want = block(*args)                          # an open level alone refuses nothing
        args[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(NotImplementedError, match="jvp"):
            block(*args)
    assert torch.equal(want, forward(*operands()))


def test_without_gradients_the_call_is_the_kernels_own(block):
    x, wg, wu = operands()
    wg.requires_grad_()
    with torch.no_grad():
        a = block(x, wg, wu)
    assert a.grad_fn is None and not a.requires_grad
    with torch.inference_mode():
        assert torch.equal(block(x, wg, wu), a)
