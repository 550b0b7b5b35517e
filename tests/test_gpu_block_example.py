"""The example that runs the selective state space block's operators together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    path = os.path.join(ROOT, "examples")
    if path not in sys.path:
        sys.path.insert(0, path)
    import selective_block
    return selective_block


def test_tokens_continue_prompts_and_training_lowers_the_loss():
    worst, losses = _example().main(width=64, batch=3, tokens=70, new=3, steps=3)
    # bf16 roundings of six stages, each at most 2^-8
    assert worst <= 6 * 2.0 ** -8
    assert losses[-1] < losses[0]


def test_gradients_of_the_whole_block_against_differences():
    """A step along every fp32 parameter's gradient against the change of the loss."""
    ex = _example()
    block = ex.SelectiveBlock(32, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(1)
    r = torch.randn(2, 40, 32, generator=g, device="cuda")
    w = torch.randn(2, 40, 32, generator=g, device="cuda")
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        grads = block.backward(block.prompt(r)[3], w)

        def total():
            return float((block.prompt(r)[0].double() * w.double()).sum())

        for name, d in grads.items():
            p = getattr(block, name)
            v = d / d.norm()
            keep, step = p.clone(), 2.0 ** -7
            ends = []
            for sign in (1, -1):
                p.copy_(keep + sign * step * v)
                ends.append(total())
            p.copy_(keep)
            num = (ends[0] - ends[1]) / (2 * step)
            # third-order term and fp32 rounding of sums of 2560 products
            assert abs(num - float(d.norm())) <= 5e-3 * float(d.norm()), name
    finally:
        torch.backends.cuda.matmul.allow_tf32 = old
