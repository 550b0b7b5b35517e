"""The selective state space block's kernels at the ends of the number range.

Tolerances, fixed before the first run.  sigmoid(x) of a very negative x: the
exponent x log2(e) is off by |x| 2^-23, the exponential, the sum and the reciprocal by
2^-22 together, so silu and its derivative are off by (2^-18 + |x| 2^-23) of their
value while e^x is a normal number, and by 2^-119 beyond (|x| e^x < 90 * 2^-126).
A stored bf16 is off by 2^-8 of its value."""
import math

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def falcon():
    import delta_rule_attention_gb300 as m
    return m


def _gates(dtype):
    """Gates from the type's lowest value to 50, as the type holds them."""
    low = torch.finfo(dtype).min
    v = [low, low / 2, -1e38, -1e37, -1e35, -1e30, -1e20, -1e10, -1e5, -1000.0, -150.0, -104.0,
         -89.0, -88.0, -87.0, -60.0, -20.0, -1.0, 0.0, 1.0, 20.0, 50.0, 0.5, -0.5]
    return torch.tensor(v, dtype=torch.float64).to(dtype)


def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    s = torch.sigmoid(v)
    return s + v * s * (1 - s)


def _close(got, want, x, dtype, name):
    """Element by element; x the silu's argument behind each element."""
    got, want, x = ref.f64(got), ref.f64(want), ref.f64(x)
    rel = 2.0 ** -18 + x.abs().clamp(max=90.0) * 2.0 ** -23 + (2.0 ** -8 if dtype == BF16 else 0.0)
    off = (got - want).abs()
    assert bool((off <= rel * want.abs() + 2.0 ** -119).all()), (name, got, want)


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_silu_over_the_whole_range(dtype, odd):
    """Filters that pass the newest input, so that the silu's argument is x itself."""
    v = _gates(dtype)
    C = v.numel() - odd
    x = torch.stack([v.roll(k)[:C] for k in range(11)])[None]  # [1, 11, C]
    w = torch.zeros(C, 2)
    w[:, 1] = 1.0
    m, xc, wc = falcon(), x.cuda(), w.cuda()
    y, _ = m.falcon_short_conv_fwd(xc, wc)
    x64 = ref.f64(x)
    _close(y, _silu(x64), x64, dtype, "y")
    g = m.falcon_short_conv_bwd(xc, wc, torch.ones_like(xc))
    _close(g["dx"], _dsilu(x64), x64, dtype, "dx")
    st = torch.zeros(11, 1, C, dtype=dtype, device="cuda")
    one = m.falcon_short_conv_step(xc[0], wc, st)
    _close(one, _silu(x64[0]), x64[0], dtype, "step")


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_gate_over_the_whole_range(dtype, odd):
    v = _gates(dtype)
    D, T, N = v.numel() - odd, 35, 16
    g = torch.Generator().manual_seed(1)
    z = torch.stack([v.roll(k)[:D] for k in range(T)])[None]
    u, delta = (torch.randn(1, T, D, generator=g).to(dtype) for _ in range(2))
    Bm, Cm = (torch.randn(1, T, 1, N, generator=g).to(dtype) for _ in range(2))
    A = -torch.exp(torch.randn(D, N, generator=g))
    dy = torch.randn(1, T, D, generator=g).to(dtype)
    d = dict(u=u, delta=delta, A=A, Bm=Bm, Cm=Cm, z=z, D=torch.randn(D, generator=g))
    c = {k: t.cuda() for k, t in d.items()}
    m = falcon()
    y, _ = m.falcon_selective_scan_fwd(**c)
    got = m.falcon_selective_scan_bwd(**c, dy=dy.cuda())
    h = torch.zeros(T, D, N, device="cuda")
    rows = {k: c[k][0] for k in ("u", "delta", "Bm", "Cm", "z")}
    one = m.falcon_selective_scan_step(rows["u"], rows["delta"], c["A"], rows["Bm"], rows["Cm"], h,
                                       D=c["D"], z=rows["z"])
    r = {k: ref.f64(t) for k, t in d.items()}
    # ||err|| / ||ref|| of a scan of T tokens, and of its gates (no argument with a
    # value to speak of is below -60)
    tol = (T + 16) * 2.0 ** -21 + 60 * 2.0 ** -23 + (2.0 ** -8 if dtype == BF16 else 0.0)
    assert ref.rel(y, ref.scan(**r)[0]) <= tol
    grads = ref.gradients(ref.scan, r, [ref.f64(dy), None])
    for mine, theirs in (("du", "u"), ("ddelta", "delta"), ("dz", "z"), ("dB", "Bm"), ("dC", "Cm"),
                         ("dA", "A"), ("dD", "D")):
        assert ref.rel(got[mine], grads[theirs]) <= tol, mine
    want = ref.scan(**{**r, **{k: r[k].transpose(0, 1) for k in rows}})[0][:, 0]
    assert ref.rel(one, want) <= tol
    # a gate far below zero closes
    shut = z[0] < -200
    assert float(y[0][shut.cuda()].abs().max()) <= 2.0 ** -119
    assert float(one[shut.cuda()].abs().max()) <= 2.0 ** -119
    assert float(got["dz"][0][shut.cuda()].abs().max()) <= 2.0 ** -119
