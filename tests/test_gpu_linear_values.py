"""Values out of the ordinary: how far a NaN or an infinity of one token reaches, and rows
whose squares leave float32."""
import pytest
import torch

from test_gpu_linear import BF16, F32, decay_case, falcon, gen, no_timeout, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [60, 700])
def test_one_bad_token_stays_in_its_head(falcon, T, bad, name, dtype):  # noqa: F811
    """Its own output is no number; what lies 128 tokens before it, in another head or in
    another row is as it was.  The gradient's adjoint runs the other way."""
    B, H, m = 2, 3, 64
    c = decay_case(B, H, T, m, m, dtype, seed=T)
    c["dO"], c["dS_T"] = randn(gen(1), B, H, T, m, dtype=dtype), randn(gen(2), B, H, m, m)
    at = T // 2 + 3
    dirty = {**c, name: c[name].clone()}
    dirty[name][1, 2, at, 5] = bad

    def run(c):
        fwd = {n: t for n, t in c.items() if n not in ("dO", "dS_T")}
        o, S = falcon.falcon_decay_attn_fwd(**fwd)
        return dict(falcon.falcon_decay_attn_bwd(**c), o=o, S=S)

    want, got = run(c), run(dirty)
    for n, t in want.items():
        rest = torch.ones(B, H, dtype=torch.bool, device="cuda")
        rest[1, 2] = False
        assert torch.equal(got[n][rest], t[rest]), n
    last = max(at - 128, 0)
    assert torch.equal(got["o"][1, 2, :last], want["o"][1, 2, :last])
    assert not torch.isfinite(got["o"][1, 2, at]).all()
    if name == "q":
        assert torch.equal(got["S"], want["S"]) and torch.equal(got["dq"], want["dq"])
    else:
        assert not torch.isfinite(got["S"][1, 2]).all()
        assert torch.equal(got["dS0"], want["dS0"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,m", [(1, 64), (3, 64), (2, 111), (1, 4096)])
@pytest.mark.parametrize("large", [3e19, 3e38])
def test_rows_whose_squares_leave_float32(falcon, large, H, m, dtype):  # noqa: F811
    """Counted as infinitely large: what is normalised is zero, and nothing is NaN, not where
    the gradient's own sums leave float32 too."""
    B, T = 2, 5
    D = H * m
    h = randn(gen(1), B, H, T, m, dtype=dtype)
    h[1, H - 1, 3] = torch.tensor([large, -1e25], device="cuda").to(dtype).repeat(m)[:m]
    x, z, d, e = (randn(gen(i), B, T, D, dtype=dtype) for i in range(2, 6))
    x[0, 2] = large
    w = randn(gen(7), D)
    out, nxt = falcon.falcon_gated_norm_fwd(h, weight=w, z=z, scale=w, x=x, next_weight=w)
    assert torch.isfinite(out).all() and torch.isfinite(nxt).all()
    assert torch.equal(out[1, 3, D - m:], x[1, 3, D - m:])
    assert (nxt[0, 2] == 0).all() and (nxt[1, 3] != 0).any()
    g = falcon.falcon_gated_norm_bwd(h, d, dnext=e, out=out, weight=w, z=z, scale=w,
                                     next_weight=w)
    assert all(torch.isfinite(t).all() for t in g.values())
    assert (g["dh"][1, H - 1, 3] == 0).all() and (g["dz"][1, 3, D - m:] == 0).all()
    assert torch.equal(g["dx"][0, 2], d[0, 2])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_zeros_beside_the_smallest_stabiliser(falcon, dtype):  # noqa: F811
    """1 / eps leaves float32, 1 / sqrt(eps) does not: rows of zeros stay zeros, and so do
    their gradients' second parts."""
    B, T, D, eps = 1, 6, 64, 1e-40
    h = torch.zeros(B, T, D, dtype=dtype, device="cuda")
    h[0, 3:] = randn(gen(1), 3, D, dtype=dtype)
    d, w = randn(gen(2), B, T, D, dtype=dtype) * 1e-3, randn(gen(3), D)
    out, nxt = falcon.falcon_gated_norm_fwd(h, weight=w, next_weight=w, eps=eps)
    assert (out[0, :3] == 0).all() and (nxt[0, :3] == 0).all()
    g = falcon.falcon_gated_norm_bwd(h, d, dnext=d, out=out, weight=w, next_weight=w, eps=eps,
                                     residual=False)
    r = torch.rsqrt(torch.tensor(eps, dtype=torch.float32).double()).cuda()
    # dnext comes back through both norms of a row of zeros: d w r, then w r again
    want = (d[0, :3].double() + d[0, :3].double() * w * r) * w * r
    within = want.abs() < 3e38
    off = (g["dh"][0, :3].double() - want).abs()
    assert (off[within] <= (2.0 ** -8 if dtype is BF16 else 2.0 ** -20) * 1.02 * want.abs()[within]).all()
    assert all(torch.isfinite(g["dh"][0, 3:]).flatten()) and torch.isfinite(g["dweight"]).all()
    assert torch.isfinite(g["dnext_weight"]).all()
