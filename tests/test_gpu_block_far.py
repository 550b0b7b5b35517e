"""Elements more than 2^31 (and 2^32 bytes) behind a tensor's first: pools of states with
many slots, and rows with long strides.

Tolerances as in test_gpu_block.py."""
import pytest
import torch

import block_reference as ref
import block_vectorised as vec

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def falcon():
    import delta_rule_attention_gb300 as m
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def test_tokens_of_far_slots():
    m, g = falcon(), _gen(0)
    C, W, D, S, N = 4096, 4, 2048, 16, 5
    x, w = torch.randn(N, C, generator=g, device="cuda").to(BF16), \
        torch.randn(C, W, generator=g, device="cuda")
    pool = (1 << 31) // ((W - 1) * C) + 7
    state = torch.zeros(pool, W - 1, C, dtype=BF16, device="cuda")
    slots = torch.tensor([pool - 1, 0, pool - 3, 1, pool // 2], dtype=torch.int32, device="cuda")
    state[slots.long()] = torch.randn(N, W - 1, C, generator=g, device="cuda").to(BF16)
    old = state[slots.long()].clone()
    y = m.falcon_short_conv_step(x, w, state, slots=slots)
    want, tail = ref.conv(ref.f64(x)[:, None], ref.f64(w), state=ref.f64(old))
    assert ref.rel(y, want[:, 0]) <= 2.0 ** -18 + 2.0 ** -8
    assert torch.equal(ref.f64(state[slots.long()]), tail)
    del state

    pool = (1 << 31) // (D * S) + 7
    h = torch.zeros(pool, D, S, device="cuda")
    slots = torch.tensor([pool - 1, 0, pool - 3, 1, pool // 2], dtype=torch.int32, device="cuda")
    h[slots.long()] = torch.randn(N, D, S, generator=g, device="cuda")
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = dict(u=r(N, D), delta=r(N, D), A=-torch.exp(r(D, S)), Bm=r(N, 1, S), Cm=r(N, 1, S))
    before = h[slots.long()].clone()
    y = m.falcon_selective_scan_step(**d, h=h, slots=slots)
    rows = {k: ref.f64(v) if k == "A" else ref.f64(v)[:, None] for k, v in d.items()}
    want, hn = ref.scan(**rows, h0=ref.f64(before))
    assert ref.rel(y, want[:, 0]) <= 17 * 2.0 ** -21
    assert ref.rel(h[slots.long()], hn) <= 17 * 2.0 ** -21


@pytest.mark.parametrize("C,first", [(40, 0), (7, 3)])
def test_rows_with_long_strides(C, first):
    """Tokens 32768 elements apart, so that the last lie beyond 2^31 elements."""
    m, g = falcon(), _gen(1)
    T, stride, N = 70001, 32768, 16
    rows = torch.empty(1, T, stride, dtype=BF16, device="cuda")
    grad = torch.empty(1, T, stride, dtype=BF16, device="cuda")
    part = lambda t, i, n: t[..., first + 64 * i:first + 64 * i + n]  # noqa: E731
    new = lambda n: torch.randn(1, T, n, generator=g, device="cuda").to(BF16)  # noqa: E731
    for i, n in enumerate((C, C, N, N, C)):
        part(rows, i, n).copy_(new(n))
    u, delta, Bm, Cm, z = (part(rows, i, n) for i, n in enumerate((C, C, N, N, C)))
    Bm, Cm = Bm.unsqueeze(2), Cm.unsqueeze(2)
    A = -torch.exp(torch.randn(C, N, generator=g, device="cuda"))
    skip = torch.randn(C, generator=g, device="cuda")
    w = torch.randn(C, 4, generator=g, device="cuda")
    dy = new(C)
    # the same tensors close together give the same results, up to what vector and
    # single accesses add in another order
    near = {k: v.contiguous() for k, v in dict(u=u, delta=delta, Bm=Bm, Cm=Cm, z=z).items()}
    far = dict(u=u, delta=delta, Bm=Bm, Cm=Cm, z=z)
    y, h = m.falcon_selective_scan_fwd(**near, A=A, D=skip)
    yf, hf = m.falcon_selective_scan_fwd(**far, A=A, D=skip, y=part(grad, 0, C))
    assert ref.rel(yf, y) <= 2.0 ** -7 and ref.rel(hf, h) <= 2.0 ** -10
    a = m.falcon_selective_scan_bwd(**near, A=A, D=skip, dy=dy)
    part(grad, 1, C).copy_(dy)
    b = m.falcon_selective_scan_bwd(**far, A=A, D=skip, dy=part(grad, 1, C))
    for k in a:
        if a[k] is not None:
            assert ref.rel(b[k], a[k]) <= 2.0 ** -7, k
    y, tail = m.falcon_short_conv_fwd(near["u"], w)
    yf, tf = m.falcon_short_conv_fwd(u, w, y=part(grad, 2, C))
    assert torch.equal(y, yf) and torch.equal(tail, tf)
    want = vec.conv_gradients(near["u"].double(), w.double(), dy.double())
    got = m.falcon_short_conv_bwd(u, w, part(grad, 1, C), grads=dict(dx=part(grad, 3, C)))
    for k in ("dx", "dweight", "dbias"):
        tol = 2.0 ** -17 + (2.0 ** -8 if k == "dx" else 0.0)
        assert float((got[k].double() - want[k]).norm() / want[k].norm()) <= tol, k
