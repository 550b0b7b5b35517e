"""Attention with a decay against the 64-bit forms, by the size of a head's results, which
sees what an element's worst case does not: a slow head's carried state, a wrong rate.

Bounds.  A rounding to bf16 is off by at most 2^-8 of a value, evenly spread: 2^-8 / sqrt(3) =
2.3e-3 of the norm at most.  An output is a sum of independent terms, each rounded once
(a weighted q k, or the state read), and is rounded once itself: 3.2e-3, and 5e-3 leaves room
for what few values scatter.  fp32: sums of 2^-24 a term that add up like the terms
themselves, over at most 4096 of them, 2^-24 64 = 4e-6, and the weights' 2^-23 of an
exponent of up to 16: 1e-5.
"""
import pytest
import torch

import linear_reference as ref

BF16, F32 = torch.bfloat16, torch.float32
BOUND = {BF16: 5e-3, F32: 1e-5}
RATES = [0.0, -2.0 ** -11.5, -2.0 ** -9, -0.01, -0.05, -0.3]


@pytest.fixture(scope="module")
def falcon():
    import delta_rule_attention_gb300 as falcon
    yield falcon
    assert falcon.falcon_sync_check() == 0


def off_by_head(got, want):
    """||got - want|| / ||want|| of every head: [H]."""
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    dims = [d for d in range(want.dim()) if d != 1]
    return ((got - want).square().sum(dims) / want.square().sum(dims).clamp(min=1e-300)).sqrt()


def case(T, m, dv, dtype, device, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    H = len(RATES)
    c = dict(q=r(1, H, T, m), k=r(1, H, T, m), v=r(1, H, T, dv), dO=r(1, H, T, dv))
    c = {n: t.to(dtype).to(device) for n, t in c.items()}
    return c, torch.tensor(RATES, device=device)


def held(got, want, dtype, T, what):
    for part, at in (("all", slice(None)), ("first", slice(0, 128)), ("last", slice(-128, None))):
        off = off_by_head(got[:, :, at], want[:, :, at])
        assert float(off.max()) <= BOUND[dtype], (what, part, off.tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,m,dv", [(300, 128, 128), (3000, 64, 64), (700, 64, 128), (700, 128, 64)])
def test_size_of_the_error(falcon, T, m, dv, dtype):
    c, ld = case(T, m, dv, dtype, "cuda", seed=T)
    dO = c.pop("dO")
    o, S = falcon.falcon_decay_attn_fwd(**c, log_decay=ld)
    want, want_S = ref.decay_forward(**c, log_decay=ld)
    held(o, want, dtype, T, "o")
    assert float(off_by_head(S, want_S).max()) <= BOUND[F32]
    got = falcon.falcon_decay_attn_bwd(**c, log_decay=ld, dO=dO)
    want = ref.decay_gradient(**c, log_decay=ld, dO=dO)
    for name in ("dq", "dk", "dv"):
        held(got[name], want[name], dtype, T, name)
    assert float(off_by_head(got["dS0"], want["dS0"]).max()) <= BOUND[F32]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads", [1, 40])
@pytest.mark.parametrize("T,m,dv", [(640, 64, 64), (640, 128, 128), (1500, 64, 128)])
def test_carried_state_alone(falcon, T, m, dv, dtype, heads):
    """Keys and values in the first 128 tokens, queries behind them: every output is a read
    of the state that was carried there.  The gradient likewise: queries and the outputs'
    gradients in the last 128 tokens, keys and values before."""
    c, ld = case(T, m, dv, dtype, "cuda", seed=m)
    dO = c.pop("dO")
    wide = lambda t: t.repeat(1, heads, *[1] * (t.dim() - 2)) if t.dim() > 1 else t.repeat(heads)  # noqa: E731
    early, late = {n: t.clone() for n, t in c.items()}, {n: t.clone() for n, t in c.items()}
    early["k"][:, :, 128:], early["v"][:, :, 128:], early["q"][:, :, :128] = 0, 0, 0
    o, _ = falcon.falcon_decay_attn_fwd(**{n: wide(t) for n, t in early.items()},
                                        log_decay=wide(ld))
    want, _ = ref.decay_forward(**early, log_decay=ld)
    end = T - 128
    late["k"][:, :, end:], late["v"][:, :, end:] = 0, 0
    late["q"][:, :, :end], dO[:, :, :end] = 0, 0
    got = falcon.falcon_decay_attn_bwd(**{n: wide(t) for n, t in late.items()}, log_decay=wide(ld),
                                       dO=wide(dO))
    grads = ref.decay_gradient(**late, log_decay=ld, dO=dO)
    for name, a, b, span in (("o", o, want, range(128, T, 128)),
                             ("dk", got["dk"], grads["dk"], range(0, end, 128)),
                             ("dv", got["dv"], grads["dv"], range(0, end, 128))):
        for x in span:
            # heads with anything left of it to speak of
            part = b[:, :, x:x + 128]
            live = part.square().sum((0, 2, 3)).sqrt() > 1e-20
            off = off_by_head(a[:, :len(RATES), x:x + 128], part)[live]
            assert float(off.max()) <= BOUND[dtype], (name, x, off.tolist())
        assert torch.equal(a[:, :len(RATES)], a[:, -len(RATES):])


@pytest.mark.gpu
def test_a_long_row_of_many_heads_does_not_drift(falcon):
    """Heads enough for one run a row, nothing decays, and sums of one sign, so that what the
    tensor cores cut off adds up: 16 additions a chunk onto the state (of 8 tokens each), each
    by at most a step of fp32 (2^-23), over a run of 64 chunks: 1.2e-4.  Besides, the
    state's rounding to bf16 scatters by 2.3e-3 over 64 x 64 values of every mantissa (4e-5):
    five times that."""
    H, T, m = 160, 1 << 19, 64
    g = torch.Generator(device="cuda").manual_seed(1)

    def one():
        x = torch.rand(T, m, generator=g, device="cuda") \
            * torch.exp2(torch.rand(m, generator=g, device="cuda"))
        return x.bfloat16()[None, None].expand(1, H, T, m)

    q, k, v = one(), one(), one()
    o, S = falcon.falcon_decay_attn_fwd(q, k, v, torch.zeros(H, device="cuda"))
    end = T - 128
    q, k, v = (t[0, 0].double() for t in (q, k, v))
    X = k[:end].t() @ v[:end]
    want = (q[end:] @ X + torch.tril(q[end:] @ k[end:].t()) @ v[end:]) * m ** -0.5
    for h in (0, 77, H - 1):
        got = o[0, h, end:].double()
        low = float((got * want).sum() / want.square().sum()) - 1
        assert abs(low) <= 1.2e-4 + 2e-4, low
    S_want = X + k[end:].t() @ v[end:]
    assert float((S[0, 0].double() - S_want).norm() / S_want.norm()) < 1e-6


@pytest.mark.parametrize("T", [300, 3000])
def test_the_bound_sees_a_wrong_rate(T):
    """A rate half as fast again moves every head that decays by more than the bound, and
    so does a state that is not carried."""
    c, ld = case(T, 16, 16, BF16, "cpu")
    c.pop("dO")
    want, _ = ref.decay_forward(**c, log_decay=ld)
    wrong, _ = ref.decay_forward(**c, log_decay=1.5 * ld)
    assert float(off_by_head(wrong, want)[1:].min()) > 2 * BOUND[BF16]
    assert float(off_by_head(wrong[:, :, -128:], want[:, :, -128:])[1:].min()) > 2 * BOUND[BF16]
    cut = {n: t[:, :, -128:] for n, t in c.items()}
    alone, _ = ref.decay_forward(**cut, log_decay=ld)
    assert float(off_by_head(alone, want[:, :, -128:])[:4].min()) > 2 * BOUND[BF16]
