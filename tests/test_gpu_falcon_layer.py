"""The example that runs the short convolution, Falcon-1A and the clipping together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    path = os.path.join(ROOT, "examples")
    if path not in sys.path:
        sys.path.insert(0, path)
    import falcon_layer
    old = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield falcon_layer
    torch.backends.cuda.matmul.allow_tf32 = old


@pytest.mark.parametrize("dtype,dim", [(torch.float32, 16), (torch.bfloat16, 64)])
def test_tokens_continue_prompts_and_training_lowers_the_loss(example, dtype, dim):
    worst, losses = example.main(width=64, heads=3, batch=2, tokens=130, new=3, steps=3, dim=dim,
                                 dtype=dtype)
    # fp32: what the token loop and the chunk form may differ by; bf16: the roundings of
    # four stages, 2^-8 each, and of the chunk form's operands
    assert worst <= (1e-4 if dtype == torch.float32 else 2e-2 + 4 * 2.0 ** -8)
    assert losses[-1] < losses[0]


def test_gradients_of_the_layer_against_differences(example):
    """A step along every parameter's gradient against the change of the loss."""
    layer = example.FalconLayer(32, 2, 16, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(1)
    r = torch.randn(2, 70, 32, generator=g, device="cuda")
    w = torch.randn(2, 70, 32, generator=g, device="cuda")
    grads = layer.backward(layer.prompt(r)[2], w)

    def total():
        return float((layer.prompt(r)[0].double() * w.double()).sum())

    for name, d in grads.items():
        p = getattr(layer, name)
        v = d / d.norm()
        keep, step = p.clone(), 2.0 ** -8
        ends = []
        for sign in (1, -1):
            p.copy_(keep + sign * step * v)
            ends.append(total())
        p.copy_(keep)
        num = (ends[0] - ends[1]) / (2 * step)
        # third-order term (step^2 = 1.5e-5 of it) and fp32 rounding of sums of 4480 products
        assert abs(num - float(d.norm())) <= 5e-3 * float(d.norm()), name
