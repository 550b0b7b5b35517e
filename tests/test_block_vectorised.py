"""The vectorised float64 forms against the token-by-token reference (CPU)."""
import pytest
import torch

import block_reference as ref
import block_vectorised as vec


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("ragged", [False, True])
def test_conv_gradients(ragged, W, silu):
    g = torch.Generator().manual_seed(W)
    B, T, C = 4, 9, 3
    r = dict(x=_rand(g, B, T, C), weight=_rand(g, C, W), bias=_rand(g, C),
             state=_rand(g, B, W - 1, C),
             lengths=torch.tensor([9, 0, 1, 5], dtype=torch.int32) if ragged else None)
    dy, dso = _rand(g, B, T, C), _rand(g, B, W - 1, C)
    act = "silu" if silu else "identity"
    want = ref.gradients(lambda **k: ref.conv(**k, activation=act), r, [dy, dso])
    got = vec.conv_gradients(r["x"], r["weight"], dy, r["bias"], r["state"], r["lengths"], dso, silu)
    for mine, theirs in (("dx", "x"), ("dweight", "weight"), ("dbias", "bias"), ("dstate", "state")):
        assert torch.allclose(got[mine], want[theirs], rtol=1e-11, atol=1e-12), mine


@pytest.mark.parametrize("full", [True, False])
def test_scan_gradients(full):
    g = torch.Generator().manual_seed(5)
    B, T, D, G, N = 4, 7, 6, 2, 3
    r = dict(u=_rand(g, B, T, D), delta=_rand(g, B, T, D), A=-_rand(g, D, N).abs(),
             Bm=_rand(g, B, T, G, N), Cm=_rand(g, B, T, G, N))
    dh = None
    if full:
        r.update(D=_rand(g, D), z=_rand(g, B, T, D), delta_bias=_rand(g, D), h0=_rand(g, B, D, N),
                 lengths=torch.tensor([7, 0, 1, 4], dtype=torch.int32))
        dh = _rand(g, B, D, N)
    dy = _rand(g, B, T, D)
    want = ref.gradients(ref.scan, r, [dy, dh])
    got = vec.scan_gradients(**r, dy=dy, dh_T=dh)
    for mine, theirs in (("du", "u"), ("ddelta", "delta"), ("dz", "z"), ("dB", "Bm"), ("dC", "Cm"),
                         ("dA", "A"), ("dD", "D"), ("ddelta_bias", "delta_bias"), ("dh0", "h0")):
        if theirs in want:
            assert torch.allclose(got[mine], want[theirs], rtol=1e-11, atol=1e-12), mine
