"""The state that enters a call, alone: keys and values (of the gradient: queries and the
outputs' gradients) of zero, so that what is left of it after the call's tokens is all
there is, however little.

Tolerances.  gamma^n X passes one multiplication for each run of tokens, of at least 64, and its
factor's exponential: 2 units in the last place and the product's half.  An exponent g n is
rounded once, by 2^-24 of itself, and those of a row's runs add up to g T.  A result below
2^-126 is off by half of 2^-149 a multiplication instead.
"""
import pytest
import torch

import linear_reference as ref
from test_gpu_linear import BF16, F32, HALF, falcon, gen, near, no_timeout, randn  # noqa: F401

pytestmark = pytest.mark.gpu
RATES = (-0.02, -0.05, -0.1, -0.2, -1.0, -1e-3)


def same_left(got, X, g, n, steps):
    x = g.double().cpu()[None, :, None, None] * torch.tensor(n, dtype=torch.float64)[
        :, None, None, None]
    want = X.double().cpu() * torch.exp(x)
    tol = want.abs() * (x.abs() * 2.0 ** -24 + steps * 2.5 * 2.0 ** -23) + steps * 2.0 ** -149
    assert ((got.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m,dv", [(64, 64), (128, 128), (37, 64)])
@pytest.mark.parametrize("T", [1, 64, 65, 128, 129, 768, 2048])
@pytest.mark.parametrize("heads", [1, 40])
def test_entering_state_alone(falcon, T, m, dv, dtype, heads):  # noqa: F811
    """With heads enough for rows of one run, and few heads for rows of many."""
    B, H = 4, heads * len(RATES)
    g = torch.tensor(RATES * heads, device="cuda")
    q, k = (randn(gen(T + i), B, H, T, m, dtype=dtype) for i in range(2))
    v = randn(gen(T + 2), B, H, T, dv, dtype=dtype)
    S0, dS = randn(gen(3), B, H, m, dv), randn(gen(4), B, H, m, dv)
    n = [T, T // 2, 0, T]
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    steps = T // 64 + 2
    o, S = falcon.falcon_decay_attn_fwd(q, k, torch.zeros_like(v), g, S0=S0, lengths=lengths)
    same_left(S, S0, g, n, steps)
    d = falcon.falcon_decay_attn_bwd(q, k, v, g, torch.zeros_like(v), S0=S0, lengths=lengths,
                                     dS_T=dS)
    same_left(d["dS0"], dS, g, n, steps)
    # outputs: scale gamma^(t+1) S0^T q, and dk = gamma^(n-1-t) dS_T v, dv likewise with k
    t = torch.arange(T, device="cuda", dtype=torch.float64)
    left = lengths.double()[:, None] - 1 - t
    on = (left >= 0)[:, None, :, None]
    grown = torch.exp(g.double()[:, None] * (t + 1))[None, :, :, None]
    left = torch.exp(g.double()[None, :, None] * left[:, None])[..., None]
    rms = m ** -0.5
    for got, f, a, X, turn in ((o, grown * rms, q, S0, False), (d["dk"], left, v, dS, True),
                               (d["dv"], left, k, dS, False)):
        X = X.double().transpose(2, 3) if turn else X.double()
        want = torch.where(on, f * (a.double() @ X), 0.0)
        size = torch.where(on, f * (a.double().abs() @ X.abs()), 0.0)
        tol = HALF[dtype] * (want.abs() + size) * 1.01 + 2.0 ** -23 * (m + T + 256) * size
        # powers below 2^-126 may count as zero
        tol = tol + 2.0 ** -126 * (a.double().abs() @ X.abs())
        assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_terms_after_a_large_state(falcon, dtype):  # noqa: F811
    """A state 2^40 times the size of what comes after it, and long forgotten."""
    B, H, T, m = 1, 4, 700, 64
    g = torch.tensor([-0.2, -0.12, -0.3, -0.7], device="cuda")
    q, k, v = (randn(gen(i), B, H, T, m, dtype=dtype) for i in range(3))
    S0 = randn(gen(3), B, H, m, m) * 2.0 ** 40
    o, S = falcon.falcon_decay_attn_fwd(q, k, v, g, S0=S0)
    want, want_S = ref.decay_forward(q, k, v, g, S0)
    size, size_S = ref.decay_forward_size(q, k, v, g, S0)
    near(o, want, size, HALF[dtype], m + T + 256, "o")
    near(S, want_S, size_S, 0.0, T + 256, "S")


def rounded_rates(n):
    """n rates near -1e-4, -2e-4, ... whose gamma lies close to the middle between two floats."""
    out = []
    for i in range(n):
        g = -1e-4 * (1 + i) - 1e-8 * torch.arange(400, dtype=torch.float32)
        gamma = torch.exp(g.double())
        off = (gamma.float().double() - gamma).abs()
        out.append(g[off.argmax()])
    return torch.stack(out).cuda()


def test_states_that_lose_a_little_token_by_token(falcon):  # noqa: F811
    """4096 tokens that add nothing.  A token rounds a state's value by at most half a step of
    it, either way: the mean over 64 x 64 values stays within 2^-24 of a step, 64 / 64 of them
    (4096 tokens, 4096 values) and five times that; what a token loses, 4e-4 at most, is off
    by 2^-23 of itself: 2e-7.  gamma rounded would be off by up to 2^-25 a token: 1.2e-4."""
    H, m, N = 4, 64, 4096
    g = rounded_rates(H)
    S0 = randn(gen(1), 1, H, m, m)
    S = S0.clone()
    zero = torch.zeros(1, H, m, device="cuda")
    q = randn(gen(2), 1, H, m)
    for _ in range(N):
        falcon.falcon_decay_attn_step(q, zero, zero, g, S)
    left = torch.exp(N * g.double())[:, None, None]
    off = S[0].double() / (S0[0].double() * left) - 1
    assert float(off.mean((1, 2)).abs().max()) <= 5 * 2.0 ** -24 + 2e-7 + 2.0 ** -24
    assert float(off.abs().max()) <= N * 2.0 ** -24
    # and one prompt of as many tokens leaves the same
    _, P = falcon.falcon_decay_attn_fwd(*(torch.zeros(1, H, N, m, device="cuda"),) * 3, g, S0=S0)
    assert float((P[0].double() / (S0[0].double() * left) - 1).abs().max()) <= 1e-5
