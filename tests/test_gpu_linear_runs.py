"""Attention with a decay over the ways in which rows are split: blocks of few and of many
chunks, many heads, calls one behind another."""
import pytest
import torch

import linear_reference as ref
from test_gpu_linear import (BF16, F32, HALF, decay_case, falcon, gen, near, once,  # noqa: F401
                             no_timeout, randn)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_blocks_of_few_and_many_chunks(falcon, m, dv):  # noqa: F811
    """Rings of barriers that are used not at all, once, as often as they have stages, and
    more often, by calls that follow one another without a pause."""
    for B, H, T, lengths in ((1, 1, 65, None), (1, 2, 128, None), (1, 1, 129, None),
                             (2, 1, 300, [300, 0]), (1, 160, 500, None), (2, 80, 400, [129, 400])):
        c = decay_case(B, H, T, m, dv, BF16, seed=T, lengths=lengths)
        dO = randn(gen(T), B, H, T, dv, dtype=BF16)
        calls = [(falcon.falcon_decay_attn_fwd(**c), falcon.falcon_decay_attn_bwd(**c, dO=dO))
                 for _ in range(6)]
        (o, S), g = calls[0]
        for (o1, S1), g1 in calls[1:]:
            assert torch.equal(o, o1) and torch.equal(S, S1)
            assert all(torch.equal(g[n], g1[n]) for n in g)
        hs = slice(0, H, max(1, H // 2))
        one = {n: t[:, hs] if n in ("q", "k", "v", "S0") else t[hs] if n == "log_decay" else t
               for n, t in c.items()}
        want, want_S = ref.decay_forward(**one)
        size, size_S = ref.decay_forward_size(**one)
        near(o[:, hs], want, size, HALF[BF16], m + T + 256, "o")
        near(S[:, hs], want_S, size_S, 0.0, T + 256, "S")
        want = ref.decay_gradient(**one, dO=dO[:, hs])
        size = ref.decay_gradient_size(**one, dO=dO[:, hs])
        for name in ("dq", "dk", "dv"):
            near(g[name][:, hs], want[name], size[name], HALF[BF16], m + dv + T + 256, name)


def test_norm_of_a_row_of_as_many_tokens_as_there_may_be(falcon):  # noqa: F811
    """One row of 2^31 - 1 tokens of a channel each: the last block's rows lie partly behind it."""
    T, eps = 2 ** 31 - 1, 0.5
    h = torch.empty(1, T, 1, dtype=BF16, device="cuda").normal_(generator=gen(1))
    room = torch.full((1, T + 512, 1), 7.0, dtype=BF16, device="cuda")
    out = room[:, 256:-256]
    w = torch.tensor([0.75], device="cuda")

    def n(at):
        x = h[0, at].double().cpu()
        return x, 0.75 * x / torch.sqrt(x * x + eps), 0.75 * eps / (x * x + eps) ** 1.5

    falcon.falcon_gated_norm_fwd(h, weight=w, eps=eps, out=out)
    parts = [slice(a, a + 100000) for a in (0, 2 ** 30, T - 100000)]
    for at in parts:
        off = (out[0, at].double().cpu() - n(at)[1]).abs()
        assert (off <= n(at)[1].abs() * (HALF[BF16] * 1.01 + 2.0 ** -18)).all()
    dout = out.clone()
    g = falcon.falcon_gated_norm_bwd(h, dout, weight=w, eps=eps, residual=False,
                                     grads=dict(dh=out))
    assert g["dh"] is out
    for at in parts:
        x, _, slope = n(at)
        d = dout[0, at].double().cpu()
        # dh = r (d w - x^2 r^2 d w): terms of the size r |d w|, at most (1 + x^2 / eps) of dh
        size = 0.75 * d.abs() / torch.sqrt(x * x + eps)
        off = (out[0, at].double().cpu() - d * slope).abs()
        assert (off <= (d * slope).abs() * HALF[BF16] * 1.01 + 2.0 ** -18 * size).all()
    assert (room[:, :256] == 7).all() and (room[:, -256:] == 7).all()


@pytest.mark.parametrize("m,dv", [(64, 64), (64, 128), (128, 64)])
def test_keys_gradient_beside_values_off_their_boundary(falcon, m, dv):  # noqa: F811
    """Only dv lies where TMA cannot be used: dk takes the tensor cores all the same.  The
    gradient of the state in place forms dk's states by themselves too: the same bits."""
    B, H, T = 2, 3, 700
    c = decay_case(B, H, T, m, dv, BF16, seed=1, lengths=[T, 300])
    dO, dS = randn(gen(2), B, H, T, dv, dtype=BF16), randn(gen(3), B, H, m, dv)
    odd = torch.empty(B, H, T, dv + 1, dtype=BF16, device="cuda")[..., 1:]
    got = falcon.falcon_decay_attn_bwd(**c, dO=dO, dS_T=dS, grads=dict(dv=odd))
    held = dS.clone()
    alone = falcon.falcon_decay_attn_bwd(**c, dO=dO, dS_T=held, grads=dict(dS0=held))
    assert torch.equal(got["dk"], alone["dk"]) and torch.equal(got["dq"], alone["dq"])
    want = ref.decay_gradient(**c, dO=dO, dS_T=dS)
    size = ref.decay_gradient_size(**c, dO=dO, dS_T=dS)
    for name in ("dq", "dk", "dv"):
        near(got[name], want[name], size[name], HALF[BF16], m + dv + T + 256, name)
    near(got["dS0"], want["dS0"], size["dS0"], 0.0, T + 256, "dS0")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 1024, 4096])
def test_norms_of_few_and_of_many_rows_one_behind_another(falcon, D, dtype):  # noqa: F811
    """Blocks that take fewer rows than they copy ahead, as many, and more, in calls that follow
    one another without a pause: the same bits, and each row what it is by itself."""
    g = gen(D)
    w = randn(g, D)
    h, z, x, d = (randn(g, 1, 3000, D, dtype=dtype) for _ in range(4))
    rows = [1, 2, 151, 303, 609, 1217, 3000]
    outs = [(falcon.falcon_gated_norm_fwd(h[:, :n], weight=w, z=z[:, :n], x=x[:, :n],
                                          next_weight=w),
             falcon.falcon_gated_norm_bwd(h[:, :n], d[:, :n], dnext=z[:, :n], out=x[:, :n],
                                          weight=w, z=z[:, :n], next_weight=w))
            for _ in range(3) for n in rows]
    for i, ((y, u), gr) in enumerate(outs):
        (y0, u0), g0 = outs[i % len(rows)]
        assert torch.equal(y, y0) and torch.equal(u, u0)
        assert all(t is None or torch.equal(t, g0[n]) for n, t in gr.items())
        (want, wu), (size, su) = ref.norm_forward(h[:, :1], weight=w, z=z[:, :1], x=x[:, :1],
                                                  next_weight=w)
        once(y[:, :1], want, size, HALF[dtype], D + 64, "out")
        once(u[:, :1], wu, su, HALF[dtype], D + 64, "next")
