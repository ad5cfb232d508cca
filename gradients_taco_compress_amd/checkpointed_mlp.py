"""Example: training a pre-norm MLP block with 8-bit activation checkpoints.

    x + W2 gelu(W1 layer_norm(x) + c1) + c2

The first half is ``norm.norm_linear``: its backward pass needs only one E4M3
code per activation element and one float32 per row, where the usual layers
keep the norm's input and output.  The script trains the block on a seeded
regression problem in bf16 with both, and prints the losses, the bytes each
keeps for the backward pass and the time of a step.

    python -m gradients_taco_compress_amd.checkpointed_mlp [--rows 8192 --hidden 2560]
"""
from __future__ import annotations

import argparse


def parameters(hidden: int, width: int, seed: int, device: str = "cuda"):
    """Norm weight and bias (float32) and the two linear layers (bf16)."""
    import torch
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=gen, device=device) * std).to(torch.bfloat16)
    p = {"norm_weight": torch.ones(hidden, device=device),
         "norm_bias": torch.zeros(hidden, device=device),
         "w1": normal(width, hidden, std=hidden ** -0.5),
         "c1": torch.zeros(width, device=device, dtype=torch.bfloat16),
         "w2": normal(hidden, width, std=0.1 * width ** -0.5),
         "c2": torch.zeros(hidden, device=device, dtype=torch.bfloat16)}
    return {k: v.requires_grad_() for k, v in p.items()}


def first_half(x, p, checkpointed: bool):
    """W1 layer_norm(x) + c1, with the 8-bit checkpoint or with torch's layers."""
    import torch
    if checkpointed:
        from . import norm
        return norm.norm_linear(x, p["norm_weight"], p["norm_bias"], p["w1"], p["c1"])
    y = torch.nn.functional.layer_norm(x, x.shape[-1:], p["norm_weight"].to(x.dtype),
                                       p["norm_bias"].to(x.dtype))
    return torch.nn.functional.linear(y, p["w1"], p["c1"])


def block(x, p, checkpointed: bool):
    import torch
    a = torch.nn.functional.gelu(first_half(x, p, checkpointed))
    return x + torch.nn.functional.linear(a, p["w2"], p["c2"])


def kept_bytes(x, p, checkpointed: bool) -> int:
    """Bytes of activations that the first half keeps for its backward pass (its
    input among them where it does)."""
    import torch
    known = {t.untyped_storage().data_ptr() for t in p.values()}
    kept = {}

    def pack(t):
        if t.untyped_storage().data_ptr() not in known:
            kept[t.untyped_storage().data_ptr()] = t.untyped_storage().nbytes()
        return t
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        z = first_half(x, p, checkpointed)
    kept.pop(z.untyped_storage().data_ptr(), None)
    return sum(kept.values())


def train(rows: int, hidden: int, steps: int, checkpointed: bool, lr: float = 1.0, seed: int = 0):
    """Losses of `steps` steps of gradient descent, and milliseconds a step."""
    import torch
    p = parameters(hidden, 4 * hidden, seed)
    teacher = parameters(hidden, 4 * hidden, seed + 1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 2)
    x = torch.randn(rows, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        target = block(x, teacher, False)
    losses = []
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for step in range(steps):
        if step == 1:
            start.record()
        error = block(x, p, checkpointed).float() - target.float()
        loss = error.square().mean()
        for t in p.values():
            t.grad = None
        loss.backward()
        with torch.no_grad():
            for t in p.values():
                t -= (lr * t.grad.float()).to(t.dtype)
        losses.append(loss.detach())
    end.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(end) / (steps - 1) if steps > 1 else 0.0
    return [float(v) for v in losses], ms


def main():
    import torch
    a = argparse.ArgumentParser(description=__doc__.split("\n", 1)[0])
    a.add_argument("--rows", type=int, default=8192)
    a.add_argument("--hidden", type=int, default=2560)
    a.add_argument("--steps", type=int, default=20)
    a = a.parse_args()
    p = parameters(a.hidden, 4 * a.hidden, 0)
    x = torch.randn(a.rows, a.hidden, device="cuda").to(torch.bfloat16).requires_grad_()
    for checkpointed in (False, True):
        losses, ms = train(a.rows, a.hidden, a.steps, checkpointed)
        print(f"{'8-bit checkpoint' if checkpointed else 'torch layers':>16}: "
              f"loss {losses[0]:.5f} -> {losses[-1]:.5f}, {ms:.2f} ms a step, norm and first "
              f"linear keep {kept_bytes(x, p, checkpointed) / 2**20:.1f} MiB", flush=True)


if __name__ == "__main__":
    main()
