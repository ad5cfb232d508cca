"""Autograd through norm.rms and gated.gated in unusual graphs: outputs whose
gradient is undefined, gradients that are added to, tangents.  Every case prints its
name before it touches the GPU."""
from __future__ import annotations

import pytest
import torch

from gated_reference import BF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def norm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import gradients_taco_compress_amd.norm as norm
    return norm


def announce(msg):
    print(f"[case] {msg}", flush=True)


def leaves(*shapes):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    return [torch.empty(s, device="cuda").normal_(generator=g).to(BF).requires_grad_() for s in shapes]


class Untouched(torch.autograd.Function):
    """Passes a value on and no gradient back."""

    @staticmethod
    def forward(ctx, y):
        return y.clone()

    @staticmethod
    def backward(ctx, dy):
        return None


def test_outputs_without_gradients(norm):
    announce("rms, undefined gradients")
    x, r, w = leaves((5, 72), (5, 72), (72,))
    y, total = norm.rms(x, w, residual=r)
    (Untouched.apply(y).sum() + (x * 2).sum()).backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0)) and r.grad is None and w.grad is None
    x.grad = None
    y, total = norm.rms(x, w, residual=r)
    (Untouched.apply(y).sum() + (total * 3).sum()).backward()
    assert torch.equal(x.grad, torch.full_like(x, 3.0)) and torch.equal(r.grad, x.grad)
    assert w.grad is None or not bool(w.grad.any())


@pytest.mark.parametrize("shape", [(5, 72), (1, 5, 72)])
def test_gradients_have_memory_of_their_own(norm, shape):
    announce(f"rms, the gradients' memory, residual {list(shape)}")
    x, r, w = leaves((5, 72), shape, (72,))
    one = torch.ones(5, 72, device="cuda", dtype=BF)
    for turn in (1.0, 2.0):
        norm.rms(x, w, residual=r)[1].backward(one)
        assert bool((one == 1).all()) and bool((x.grad == turn).all()) and bool((r.grad == turn).all())
    assert len({t.untyped_storage().data_ptr() for t in (x.grad, r.grad, one)}) == 3
    x.grad = r.grad = None
    torch.autograd.backward(norm.rms(x, w, residual=r), (one, one))
    want = x.grad.clone()
    r.grad.zero_()
    assert torch.equal(x.grad, want) and bool(want.any())


@pytest.mark.parametrize("mode", [torch.no_grad, torch.enable_grad])
def test_tangents_are_refused(mode):
    """The block has no forward-mode derivative."""
    import gradients_taco_compress_amd.gated as gated
    from torch.autograd import forward_ad
    announce(f"gated, a tangent under {mode.__name__}")
    x, wg, wu = (t.detach() for t in leaves((5, 72), (40, 72), (40, 72)))
    want = gated.gated_forward(x, wg, wu)
    with mode(), forward_ad.dual_level():
        assert torch.equal(gated.gated(x, wg, wu), want)
        for i in range(3):
            args = [x, wg, wu]
            args[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(NotImplementedError, match="jvp"):
                gated.gated(*args)
