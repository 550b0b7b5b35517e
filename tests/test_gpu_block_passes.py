"""Scan gradients whose dB and dC terms are taken in several passes.

Tolerance as in test_gpu_block.py: (T + 16) 2^-21, plus 2^-8 for a stored bf16."""
import pytest
import torch

import block_vectorised as vec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,B,T,D,G,N,ragged", [
    (torch.bfloat16, 8, 300, 2048, 1, 128, True), (torch.float32, 9, 290, 2050, 2, 100, False),
    (torch.bfloat16, 64, 265, 2048, 1, 64, True)])
def test_scan_gradient_in_several_passes(dtype, B, T, D, G, N, ragged):
    import delta_rule_attention_gb300 as m
    from delta_rule_attention_gb300.block import falcon_scan_shape
    padded = 4
    while padded < N:
        padded *= 2
    wide = {4: 256, 8: 128, 16: 64, 32: 32, 64: 8, 128: 2}[padded]
    parts = (D // G + wide - 1) // wide
    all_terms = 8 * parts * B * T * G * padded
    need = m.load_library().falcon_selective_scan_bwd_workspace_bytes(
        falcon_scan_shape(B, T, D, G, N, 0, 1))
    assert all_terms > 2 << 30 and need < all_terms + 8 * B * ((T + 31) // 32) * D * padded

    g = torch.Generator(device="cuda").manual_seed(N)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = dict(u=r(B, T, D).to(dtype), delta=(0.5 * r(B, T, D)).to(dtype), A=-torch.exp(r(D, N)),
             Bm=r(B, T, G, N).to(dtype), Cm=r(B, T, G, N).to(dtype), D=r(D),
             delta_bias=r(D) - 2.0, z=r(B, T, D).to(dtype), h0=r(B, D, N), lengths=None)
    dy, dh = r(B, T, D).to(dtype), r(B, D, N)
    if ragged:
        n = torch.randint(0, T + 1, (B,), generator=g, device="cuda")
        n[0], n[1] = T, 0
        d["lengths"] = n.to(torch.int32)
    f64 = lambda t: t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t  # noqa: E731
    want = vec.scan_gradients(**{k: f64(v) for k, v in d.items()}, dy=f64(dy), dh_T=f64(dh))
    if ragged:
        for b in range(B):
            k = int(d["lengths"][b])
            for t in (d["u"], d["delta"], d["Bm"], d["Cm"], d["z"], dy):
                t[b, k:] = float("nan")
    got = m.falcon_selective_scan_bwd(**d, dy=dy, dh_T=dh)
    again = m.falcon_selective_scan_bwd(**d, dy=dy, dh_T=dh)
    for k, v in want.items():
        half = dtype == torch.bfloat16 and k in ("du", "ddelta", "dz", "dB", "dC")
        tol = (T + 16) * 2.0 ** -21 + (2.0 ** -8 if half else 0.0)
        err = float((got[k].double() - v).norm() / v.norm())
        assert err <= tol, (k, err)
        assert torch.equal(got[k], again[k]), k
