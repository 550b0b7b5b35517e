"""The linear attention block beyond the sizes of the other tests: strides past 2^31 elements,
many narrow rows, states and parameters on element boundaries, many heads."""
import pytest
import torch

import linear_reference as ref
from test_gpu_linear import BF16, F32, HALF, falcon, gen, near, no_timeout, once, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_far_apart(falcon, dtype):  # noqa: F811
    """Batches 2^31 elements apart, read and written in place in one buffer."""
    far, T, m = 2 ** 31, 200, 64
    room = torch.empty(far + 8 * T * m, dtype=dtype, device="cuda")
    part = lambda i: room.as_strided((2, 1, T, m), (far, T * m, m, 1), i * T * m)  # noqa: E731
    g = gen(1)
    for i in range(3):
        part(i).copy_(randn(g, 2, 1, T, m, dtype=dtype))
    q, k, v, o = (part(i) for i in range(4))
    ld = torch.tensor([-0.02], device="cuda")
    falcon.falcon_decay_attn_fwd(q, k, v, ld, o=o)
    want, _ = ref.decay_forward(q, k, v, ld)
    size, _ = ref.decay_forward_size(q, k, v, ld)
    near(o, want, size, HALF[dtype], m + T + 256, "o")
    grads = dict(dq=part(4), dk=part(5), dv=part(6))
    falcon.falcon_decay_attn_bwd(q, k, v, ld, o, grads=grads)
    want, size = ref.decay_gradient(q, k, v, ld, o), ref.decay_gradient_size(q, k, v, ld, o)
    for name in grads:
        near(grads[name], want[name], size[name], HALF[dtype], 2 * m + T + 256, name)
    x, out = part(1)[:, 0], part(7)[:, 0]
    w = randn(g, m)
    falcon.falcon_gated_norm_fwd(q, weight=w, z=part(2)[:, 0], x=x, out=out)
    (y, _), (sy, _) = ref.norm_forward(q, weight=w, z=part(2)[:, 0], x=x)
    once(out, y, sy, HALF[dtype], m + 64, "out")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,H,m", [(90001, 1, 64), (70000, 2, 16), (100003, 1, 8), (30000, 3, 32),
                                      (50000, 1, 24), (20000, 2, 256)])
def test_many_narrow_rows(falcon, rows, H, m, dtype):  # noqa: F811
    """Launches that hold several vectors a thread: against the same rows a few at a time."""
    g = gen(rows)
    D = H * m
    h, z, x, d, e = (randn(g, 1, rows, D, dtype=dtype) for _ in range(5))
    w, s, n = (randn(g, D) for _ in range(3))
    heads = lambda t: t.unflatten(2, (H, m)).transpose(1, 2)  # noqa: E731
    out, nxt = falcon.falcon_gated_norm_fwd(heads(h), weight=w, z=z, scale=s, x=x, next_weight=n)
    gr = falcon.falcon_gated_norm_bwd(heads(h), d, dnext=e, out=out, weight=w, z=z, scale=s,
                                      next_weight=n)
    for a in list(range(0, rows - 50, rows // 7)) + [rows - 50]:
        cut = slice(a, a + 50)
        one = dict(h=heads(h[:, cut]), weight=w, z=z[:, cut], scale=s, next_weight=n)
        (y, u), (sy, su) = ref.norm_forward(x=x[:, cut], **one)
        once(out[:, cut], y, sy, HALF[dtype], D + 64, "out")
        once(nxt[:, cut], u, su, HALF[dtype], D + 64, "next")
        want, size = ref.norm_gradient(dout=d[:, cut], dnext=e[:, cut], out=out[:, cut], **one)
        once(gr["dx"][:, cut], want["dx"], size["dx"], HALF[dtype], D + 64, "dx")
        once(gr["dz"][:, cut], want["dz"], size["dz"], HALF[dtype], D + 64, "dz")
        once(gr["dh"][:, :, cut], want["dh"], size["dh"], HALF[dtype], D + 64, "dh")
    # the parameters' gradients add over all rows
    flat = h.double().unflatten(2, (H, m))
    r = torch.rsqrt(flat.square().mean(-1, keepdim=True) + 1e-6)
    y = out.double()
    q = torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    ew = e.double() * n
    dd = d.double() + q * (ew - y * q * q * (ew * y).mean(-1, keepdim=True))
    act = z.double() * torch.sigmoid(z.double())
    terms = dd * act * (flat * r).flatten(2)
    for name, t in (("dweight", terms * s), ("dscale", terms * w), ("dnext_weight", e * y * q)):
        off = (gr[name].double() - t.sum((0, 1))).abs()
        # a term passes at most 1024 sums: those of a thread, of its block, and of the blocks
        assert (off <= 2.0 ** -23 * 1024 * t.abs().sum((0, 1))).all(), name


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,H,m", [(5000, 1, 1051), (2500, 1, 2055), (2500, 1, 4099), (2500, 1, 8191),
                                      (2500, 1, 8192), (2500, 12, 111), (2500, 11, 97),
                                      (9000, 1, 130), (2500, 2, 2048)])
def test_many_wide_rows(falcon, rows, H, m, dtype):  # noqa: F811
    """Rows that leave room for none ahead, or lie on no 16-byte boundary."""
    test_many_narrow_rows(falcon, rows, H, m, dtype)


def test_step_and_norms_off_their_boundaries(falcon):  # noqa: F811
    g = gen(3)
    N, H, m, dv = 3, 2, 64, 64
    q, k = (randn(g, N, H, m, dtype=BF16) for _ in range(2))
    v = randn(g, N, H, dv, dtype=BF16)
    ld = torch.tensor([-0.3, -1.0], device="cuda")
    flat = randn(g, N * H * m * dv + 1)
    S = flat[1:].view(N, H, m, dv)
    one = dict(q=q[:, :, None], k=k[:, :, None], v=v[:, :, None], log_decay=ld, S0=S.clone())
    out = falcon.falcon_decay_attn_step(q, k, v, ld, S)
    want, want_S = ref.decay_forward(**one)
    size, size_S = ref.decay_forward_size(**one)
    once(out[:, :, None], want, size, HALF[BF16], m + 16, "o")
    once(S, want_S, size_S, 0.0, 8, "S")
    D = 128
    w = randn(g, D + 1)[1:]
    h = randn(g, 2, 5, D, dtype=BF16)
    x = randn(g, 2, 5, D + 1, dtype=BF16)[..., 1:]
    got, nxt = falcon.falcon_gated_norm_fwd(h, weight=w, scale=w, x=x, next_weight=w)
    (y, u), (sy, su) = ref.norm_forward(h, weight=w, scale=w, x=x, next_weight=w)
    once(got, y, sy, HALF[BF16], D + 64, "out")
    once(nxt, u, su, HALF[BF16], D + 64, "next")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_heads(falcon, dtype):  # noqa: F811
    """More heads than blocks, one run each: the same heads a few at a time."""
    B, H, T, m = 7, 61, 140, 64
    g = gen(4)
    q, k, v, do = (randn(g, B, H, T, m, dtype=dtype) for _ in range(4))
    ld = -torch.exp2(-10 * torch.rand(H, generator=g, device="cuda"))
    lengths = torch.tensor([140, 1, 0, 139, 128, 129, 64], dtype=torch.int32, device="cuda")
    o, S = falcon.falcon_decay_attn_fwd(q, k, v, ld, lengths=lengths)
    d = falcon.falcon_decay_attn_bwd(q, k, v, ld, do, lengths=lengths)
    for hs in (slice(0, 2), slice(30, 32), slice(59, 61)):
        one = [t[:, hs] for t in (q, k, v)] + [ld[hs]]
        want, want_S = ref.decay_forward(*one, lengths=lengths)
        size, size_S = ref.decay_forward_size(*one, lengths=lengths)
        near(o[:, hs], want, size, HALF[dtype], m + T + 256, "o")
        near(S[:, hs], want_S, size_S, 0.0, T + 256, "S")
        want = ref.decay_gradient(*one, do[:, hs], lengths=lengths)
        size = ref.decay_gradient_size(*one, do[:, hs], lengths=lengths)
        for name in ("dq", "dk", "dv"):
            near(d[name][:, hs], want[name], size[name], HALF[dtype], 2 * m + T + 256, name)
        near(d["dS0"][:, hs], want["dS0"], size["dS0"], 0.0, T + 256, "dS0")
