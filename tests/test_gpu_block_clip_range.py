"""Clipping where the squares of the gradients leave float32.

Tolerances as in test_gpu_block.py: the norm 2^-18; an output 2^-17 of its value, plus
2^-8 for a stored bf16, plus 2^-150 / scale of the value, half float32's spacing below
its normal numbers, for a scale that is such a number, plus half the stored type's
spacing there (2^-150, bf16 2^-134)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def falcon():
    import delta_rule_attention_gb300 as m
    return m


def _grads(dtype, size):
    g = torch.Generator().manual_seed(2)
    return [(size * torch.randn(n, generator=g, dtype=torch.float64)).to(dtype).cuda()
            for n in (1, 7, 4096, 20001)]


def _check(grads, max_norm, out=None, eps=0.0):
    n = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    scale = min(1.0, max_norm / (n + eps))
    want = [t.double() * scale for t in grads]
    norm = float(falcon().falcon_clip_grad_norm(grads, max_norm, out=out, eps=eps))
    if n < 3.4e38:
        assert abs(norm - n) <= 2.0 ** -18 * n
    else:
        assert norm == math.inf
    for o, w in zip(out or grads, want):
        tol = 2.0 ** -17 + (2.0 ** -8 if o.dtype == BF16 else 0.0) + 2.0 ** -150 / scale
        least = 2.0 ** -134 if o.dtype == BF16 else 2.0 ** -150
        assert bool(((o.double() - w).abs() <= tol * w.abs() + least).all())


@pytest.mark.parametrize("size", [1e20, 1e30, 1e34, 1e-21, 1e-24, 1e-30, 1e-36])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_clip_of_sizes_whose_squares_leave_float32(dtype, size):
    _check(_grads(dtype, size), 0.5 * size)
    _check(_grads(dtype, size), 0.5 * size, out=[torch.empty_like(t) for t in _grads(dtype, 1.0)])
    _check(_grads(dtype, size), 1e4 * size)  # nothing to scale


def test_clip_of_sizes_far_apart():
    """Large, ordinary, vanishing and zero gradients in one call."""
    parts = [_grads(F32, 1e25)[3], torch.zeros(5000, device="cuda"), _grads(F32, 1.0)[2],
             _grads(BF16, 1e-30)[3], _grads(F32, 1e-30)[1]]
    _check([t.clone() for t in parts], 1e24)
    _check([t.clone() for t in parts[1:]], 2.0)
    _check([t.clone() for t in parts[3:]], 1e-30)


def test_clip_of_a_norm_beyond_float32():
    """Finite gradients whose norm is not a float32: it comes out infinite, but they are
    scaled by what it is."""
    g = torch.full((1000,), 3e38, device="cuda")
    _check([g], 1.0)


def test_clip_of_zeros():
    g = [torch.zeros(9000, device="cuda"), torch.zeros(33, dtype=BF16, device="cuda")]
    assert float(falcon().falcon_clip_grad_norm(g, 1.0)) == 0.0
    assert not g[0].any() and not g[1].any()
