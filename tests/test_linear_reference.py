"""The 64-bit forms that the linear attention block is tested against: their gradients
against differences and autograd, and their edges (no GPU needed)."""
import pytest
import torch

import linear_reference as ref

F64 = torch.float64


def _decay_case(B=2, H=2, T=5, m=3, dv=4, seed=0, ends=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    c = dict(q=r(B, H, T, m), k=r(B, H, T, m), v=r(B, H, T, dv),
             log_decay=-torch.rand(H, generator=g, dtype=F64) * 2, dO=r(B, H, T, dv))
    if ends:
        c.update(S0=r(B, H, m, dv), dS_T=r(B, H, m, dv))
    return c


@pytest.mark.parametrize("lengths", [None, [5, 2], [0, 1]])
@pytest.mark.parametrize("ends", [True, False])
def test_decay_gradient_against_differences(lengths, ends):
    c = _decay_case(ends=ends)
    grads = ref.decay_gradient(lengths=lengths, **c)

    def loss(**kw):
        a = {n: t for n, t in {**c, **kw}.items() if n not in ("dO", "dS_T")}
        o, S = ref.decay_forward(lengths=lengths, **a)
        return (o * c["dO"]).sum() + ((S * c["dS_T"]).sum() if ends else 0.0)

    step = 1e-6
    for name in ("q", "k", "v") + (("S0",) if ends else ()):
        got = grads["d" + name]
        for at in range(0, c[name].numel(), 7):
            up, down = c[name].clone(), c[name].clone()
            up.view(-1)[at] += step
            down.view(-1)[at] -= step
            want = (loss(**{name: up}) - loss(**{name: down})) / (2 * step)
            assert abs(got.reshape(-1)[at] - want) < 1e-7


def test_decay_of_one_and_of_nothing():
    c = _decay_case(H=3, ends=False)
    c["log_decay"] = torch.tensor([0.0, 5.0, -float("inf")], dtype=F64)
    o, S = ref.decay_forward(c["q"], c["k"], c["v"], c["log_decay"], scale=1.0)
    whole = torch.einsum("bhtm,bhtd->bhmd", c["k"], c["v"])
    assert torch.allclose(S[:, :2], whole[:, :2])  # a positive rate counts as none
    last = c["k"][:, 2, -1, :, None] * c["v"][:, 2, -1, None, :]
    assert torch.allclose(S[:, 2], last)


def test_a_dropped_decay_is_seen():
    c = _decay_case(ends=False)
    o, _ = ref.decay_forward(c["q"], c["k"], c["v"], c["log_decay"])
    wrong, _ = ref.decay_forward(c["q"], c["k"], c["v"], torch.zeros(2, dtype=F64))
    assert (o - wrong).abs().max() > 0.1


@pytest.mark.parametrize("gate", ["silu", "sigmoid", "identity", None])
@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("full", [True, False])
@pytest.mark.parametrize("lengths", [None, [3, 0]])
def test_norm_gradient_against_autograd(gate, heads, full, lengths):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    B, T, m, eps = 2, 4, 5, 1e-3
    D = heads * m
    h = r(B, heads, T, m) if heads > 1 else r(B, T, m)
    p = dict(h=h, weight=r(D), scale=r(D) if full else None, x=r(B, T, D) if full else None,
             z=r(B, T, D) if gate else None, next_weight=r(D) if full else None)
    p = {n: t.requires_grad_() for n, t in p.items() if t is not None}
    kind = gate or "silu"
    on = (torch.arange(T)[None, :] < torch.tensor(ref.lengths_of(lengths, B, T))[:, None])
    on = on[..., None].to(F64)

    def forward():
        hr = ref._rows(p["h"])
        y = (hr / torch.sqrt(hr.square().mean(-1, keepdim=True) + eps)).flatten(2) * p["weight"]
        if gate:
            y = y * ref._gate(p["z"], kind)[0]
        if full:
            y = p["x"] + p["scale"] * y
        y = y * on
        u = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * p["next_weight"] if full \
            else None
        return y, u

    y, u = forward()
    dout, dnext = r(B, T, D), r(B, T, D) if full else None
    loss = (y * dout).sum() + ((u * dnext).sum() if full else 0.0)
    want = dict(zip(p, torch.autograd.grad(loss, list(p.values()))))
    got, size = ref.norm_gradient(
        h, dout, dnext, y if full else None, p["weight"], p.get("z"), kind, p.get("scale"), full,
        p.get("next_weight"), lengths, eps)
    for name, t in want.items():
        assert torch.allclose(got["d" + name], t, atol=1e-10), name
        assert (size["d" + name] >= got["d" + name].abs() - 1e-12).all(), name
    (out, nxt), _ = ref.norm_forward(h, p["weight"], p.get("z"), kind, p.get("scale"), p.get("x"),
                                     p.get("next_weight"), lengths, eps)
    assert torch.allclose(out, y) and (nxt is None or torch.allclose(nxt, u))
