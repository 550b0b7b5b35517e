"""The gates of the norm and their slopes over all arguments, each against its own size."""
import pytest
import torch

import linear_reference as ref
from test_gpu_linear import BF16, F32, HALF, falcon, gen, no_timeout, once, randn  # noqa: F401

pytestmark = pytest.mark.gpu


def gate64(z, gate):
    """A gate and its slope without a difference from one: the reference's own 1 - p has
    nothing left of e^{-z} at z = 37, in 64 bits either."""
    if z is None:
        return 1.0, 0.0
    p, q = torch.sigmoid(z), torch.sigmoid(-z)
    return dict(silu=(z * p, p * (1 + z * q)), sigmoid=(p, p * q),
                identity=(z, torch.ones_like(z)))[gate]


def rounded_once(got, want, size, half, terms, what):
    """Values past the type's largest are infinite, the others as in `once`."""
    past = want.abs() > torch.finfo(got.dtype).max
    got = got.cpu()
    assert torch.equal(got[past].double(), want[past].sign() * float("inf")), what
    once(got[~past], want[~past], size[~past], half, terms, what)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", ["silu", "sigmoid", "identity"])
@pytest.mark.parametrize("m", [64, 111])
def test_gates_from_end_to_end(falcon, monkeypatch, gate, m, dtype):  # noqa: F811
    """A product of a few factors: its relative error is theirs, and the exponent's of
    e^{-z}, 2^-24 of at most 1.45 |z| halvings.  A silu's slope is a sum of two parts."""
    monkeypatch.setattr(ref, "_gate", gate64)
    B, T = 2, 40
    z = torch.cat([torch.linspace(-85, 85, B * T * m - 8, device="cuda"),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 3e38, -3e38], device="cuda")])
    z = z.to(dtype).view(B, T, m)
    h, d = randn(gen(1), B, T, m, dtype=dtype), randn(gen(2), B, T, m, dtype=dtype)
    c = dict(z=z, gate=gate, eps=1e-5)
    out, _ = falcon.falcon_gated_norm_fwd(h, **c)
    (y, _), (sy, _) = ref.norm_forward(h, **c)
    rounded_once(out, y, sy, HALF[dtype], m + 64, "out")
    got = falcon.falcon_gated_norm_bwd(h, d, residual=False, **c)
    want, size = ref.norm_gradient(h, d, residual=False, **c)
    rounded_once(got["dz"], want["dz"], size["dz"], HALF[dtype], m + 64, "dz")
    # dh takes the row's sum of d act(z) h: held where that lies in fp32's range, which it
    # leaves for the identity of 3e38 (times d h, of which some exceed 3.4e38 / 3e38)
    total = (d * h).double().cpu().abs() * gate64(z.double().cpu(), gate)[0].abs()
    rows = total.sum(-1) < 2.0 ** 127
    assert int(rows.sum()) >= B * T - 1
    rounded_once(got["dh"].cpu()[rows], want["dh"][rows], size["dh"][rows], HALF[dtype], m + 64, "dh")
