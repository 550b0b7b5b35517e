"""The linear attention block's operators as a program uses them: the example's model against
plain torch and autograd, and calls on streams, in graphs and side by side."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def falcon():
    import delta_rule_attention_gb300 as falcon
    return falcon


@pytest.fixture(scope="module")
def example():
    import decay_block
    return decay_block


def norm64(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def plain(model, x, blocks, norm_in):
    """The model's output in 64 bits."""
    u = norm64(x, norm_in)
    B, T, _ = x.shape
    gap = torch.arange(T, device=x.device)[:, None] - torch.arange(T, device=x.device)
    decay = torch.where(gap >= 0, torch.exp(model.log_decay.double()[:, None, None]
                                            * gap.clamp(min=0)), 0.0)
    for p in blocks:
        q, k, v, z = model.parts(u @ p["w_in"].T)
        o = (q @ k.transpose(-1, -2) * decay * model.dim ** -0.5) @ v
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6)
        y = o.transpose(1, 2).flatten(2) * p["norm_heads"] * torch.nn.functional.silu(z)
        x = x + norm64(y @ p["w_out"].T, p["norm_post"]) * p["scale"]
        u = norm64(x, p["norm_next"])
    return u


def test_model_and_gradients(example):
    """In fp32: every step keeps 2^-20 or so of what it sums, and a few dozen steps follow one
    another; a wrong term would be of the size of the result."""
    model = example.DecayModel(96, 3, layers=2, dim=32, dtype=F32, seed=1)
    x = torch.randn(2, 150, 96, device="cuda")
    blocks = [{n: t.double().requires_grad_() for n, t in p.items()} for p in model.blocks]
    norm_in, xx = model.norm_in.double().requires_grad_(), x.double().requires_grad_()
    want = plain(model, xx, blocks, norm_in)
    out, _, kept = model.prompt(x)
    assert float((out - want).norm() / want.norm()) < 2e-5
    d = torch.randn_like(out)
    own, grads, dx = model.backward(kept, d)
    leaves = [xx, norm_in] + [p[n] for p in blocks for n in p]
    wants = torch.autograd.grad((want * d).sum(), leaves)
    gots = [dx, own["norm_in"]] + [g[n] for g, p in zip(grads, blocks) for n in p]
    for got, w in zip(gots, wants):
        assert float((got - w).norm() / w.norm()) < 5e-5


def test_model_over_padded_prompts(example):
    """Rows of a padded batch are those of the same rows by themselves, bit for bit or close
    (the runs of tokens they are split into may differ)."""
    model = example.DecayModel(128, 2, layers=2, dim=64, dtype=F32, seed=2)
    n = [70, 200, 1]
    x = torch.randn(3, 200, 128, device="cuda")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    dirty = x.clone()
    for b in range(3):
        dirty[b, n[b]:] = float("nan")
    out, states, _ = model.prompt(dirty, lengths=lengths)
    for b in range(3):
        alone, ends, _ = model.prompt(x[b:b + 1, :n[b]])
        assert float((out[b, :n[b]] - alone[0]).abs().max()) < 1e-4
        assert (out[b, n[b]:] == 0).all()
        for S, e in zip(states, ends):
            assert float((S[b] - e[0]).norm() / e.norm()) < 1e-5


def test_example_runs(example):
    worst, losses = example.main(width=128, heads=2, batch=2, tokens=200, new=3, steps=2)
    # bf16 rows into every product: 2^-8 a rounding, a dozen of them on the way
    assert worst < 5e-2 and all(torch.isfinite(torch.tensor(losses)))


def calls(falcon, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, dtype=BF16: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    B, H, T, m = 2, 4, 700, 64
    q, k, v, do = (r(B, H, T, m) for _ in range(4))
    ld = -torch.exp2(-torch.arange(1, H + 1, device="cuda").float())
    S0 = r(B, H, m, m, dtype=F32)
    z, x = r(B, T, H * m), r(B, T, H * m)
    w = r(H * m, dtype=F32)

    def run():
        o, S = falcon.falcon_decay_attn_fwd(q, k, v, ld, S0=S0)
        gr = falcon.falcon_decay_attn_bwd(q, k, v, ld, do, S0=S0, dS_T=S0)
        y, u = falcon.falcon_gated_norm_fwd(o, weight=w, z=z, scale=w, x=x, next_weight=w)
        gn = falcon.falcon_gated_norm_bwd(o, x, dnext=z, out=y, weight=w, z=z, scale=w,
                                          next_weight=w)
        gf = falcon.falcon_decay_attn_fwd(q.float(), k.float(), v.float(), ld, S0=S0)
        return [o, S, *gr.values(), y, u, *gn.values(), *gf]
    return run


def test_calls_repeat_bit_for_bit(falcon):
    run = calls(falcon)
    first = run()
    for _ in range(3):
        for a, b in zip(first, run()):
            assert torch.equal(a, b)


def test_calls_on_streams_side_by_side(falcon):
    runs = [calls(falcon, seed) for seed in range(3)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [None] * 3
    for _ in range(4):
        for i, (run, s) in enumerate(zip(runs, streams)):
            with torch.cuda.stream(s):
                got[i] = run()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)
    assert falcon.falcon_sync_check() == 0


def test_calls_on_a_given_stream(falcon):
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(1, 2, 300, 64, generator=g, device="cuda").to(BF16) for _ in range(3))
    ld = torch.full((2,), -0.1, device="cuda")
    o, S = falcon.falcon_decay_attn_fwd(q, k, v, ld)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, S2 = falcon.falcon_decay_attn_fwd(q, k, v, ld, stream=s)
    y2, _ = falcon.falcon_gated_norm_fwd(o2, stream=s)
    d2 = falcon.falcon_decay_attn_bwd(q, k, v, ld, o2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    assert torch.equal(y2, falcon.falcon_gated_norm_fwd(o)[0])
    for a, b in zip(d2.values(), falcon.falcon_decay_attn_bwd(q, k, v, ld, o).values()):
        assert torch.equal(a, b)


def test_calls_in_graphs(falcon):
    """Two captured graphs, replayed in turn and with new inputs."""
    runs = [calls(falcon, seed) for seed in range(2)]
    want = [run() for run in runs]
    graphs, outs = [], []
    for run in runs:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for a, b in zip(o, w):
            assert torch.equal(a, b)


def test_step_in_a_graph_moves_its_states(falcon):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(3, 2, 64, generator=g, device="cuda").to(BF16) for _ in range(3))
    ld = torch.full((2,), -0.5, device="cuda")
    S = torch.zeros(3, 2, 64, 64, device="cuda")
    want = S.clone()
    for _ in range(5):
        o = falcon.falcon_decay_attn_step(q, k, v, ld, want)
    falcon.falcon_decay_attn_step(q, k, v, ld, S.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = falcon.falcon_decay_attn_step(q, k, v, ld, S)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(S, want) and torch.equal(out, o)


def test_prompt_and_steps_agree(falcon):
    """A prompt's state carries on token by token, and a split prompt's through the middle."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, H, T, m = 2, 3, 260, 64
    q, k, v = (torch.randn(B, H, T, m, generator=g, device="cuda") for _ in range(3))
    ld = torch.tensor([-1.0, -0.05, 0.0], device="cuda")
    o, S = falcon.falcon_decay_attn_fwd(q, k, v, ld)
    cut = 250
    _, P = falcon.falcon_decay_attn_fwd(q[:, :, :cut], k[:, :, :cut], v[:, :, :cut], ld)
    for t in range(cut, T):
        one = falcon.falcon_decay_attn_step(q[:, :, t], k[:, :, t], v[:, :, t], ld, P)
        assert float((one - o[:, :, t]).abs().max()) < 1e-3
    assert float((P - S).norm() / S.norm()) < 1e-6
