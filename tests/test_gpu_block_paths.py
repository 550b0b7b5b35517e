"""Paths that only larger calls take: convolution gradients that walk several blocks
of tokens and several runs a thread, scan gradients whose blocks walk several chunks,
and clipping with whole-tile chunks and passing loads.  Each case states the path
that the sizes choose, read off the workspace where it shows.

Tolerances as in test_gpu_block.py, fixed before the first run; sums over tokens add
their terms in parts of at most 1024 with float32 sums, each off by 2^-24 of the
partial sum, of which at most 2^11 follow one another: 2^-13 at the worst, and the
square root of it, 2^-18, for roundings without a common sign; twice that is asked."""
import pytest
import torch

import block_reference as ref
import block_vectorised as vec

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
CONV = 2.0 ** -17


def falcon():
    import delta_rule_attention_gb300 as m
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _draw(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _wide(d):
    return {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
            for k, v in d.items()}


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def _lengths(g, B, T):
    n = torch.randint(0, T + 1, (B,), generator=g, device="cuda")
    n[0], n[-1] = T, 0
    return n.to(torch.int32)


def _conv_run(m, B, T, C, W):
    """(tokens of a run, parts of the sums) that the library chose."""
    from delta_rule_attention_gb300.block import falcon_conv_shape
    lib = m.load_library()
    need = lib.falcon_short_conv_bwd_workspace_bytes(falcon_conv_shape(B, 1, T, C, W, 0, 1))
    parts = need // (4 * (W + 1) * C)
    runs = [r for r in range(8, 129, 8)
            if min(B * ((T + r - 1) // r), 1024) == parts]
    return runs, parts


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("B,T,C,W,run,turns", [
    (3, 1030, 1030, 4, 24, False), (16, 515, 331, 3, 24, False), (32, 515, 130, 2, 32, False),
    (40, 1030, 264, 4, 80, False), (200, 700, 6, 4, 128, True), (200, 700, 5, 3, 128, True)])
def test_conv_gradient_over_long_runs(B, T, C, W, run, turns, silu, dtype):
    """Runs of several blocks of tokens: the first, whole ones, and the row's end; `turns`:
    more runs than parts, so that a thread walks two."""
    m, g = falcon(), _gen(B + T + C + W)
    runs, parts = _conv_run(m, B, T, C, W)
    if turns:
        assert parts == 1024 < B * ((T + 127) // 128)
    else:
        assert runs == [run]
    d = dict(x=_draw(g, B, T, C, dtype=dtype), weight=_draw(g, C, W), bias=_draw(g, C),
             state=_draw(g, B, W - 1, C, dtype=dtype), lengths=_lengths(g, B, T))
    dy, dso = _draw(g, B, T, C, dtype=dtype), _draw(g, B, W - 1, C, dtype=dtype)
    want = vec.conv_gradients(**_wide(d), dy=dy.double(), dstate_out=dso.double(), silu=silu)
    for b in range(B):  # what lies behind a row's length is never used
        n = int(d["lengths"][b])
        d["x"][b, n:] = float("nan")
        dy[b, n:] = float("nan")
    got = m.falcon_short_conv_bwd(**d, dy=dy, dstate_out=dso,
                                  activation="silu" if silu else "identity")
    for k, v in want.items():
        tol = CONV + (2.0 ** -8 if dtype == BF16 and k in ("dx", "dstate") else 0.0)
        assert _rel(got[k], v) <= tol, (k, _rel(got[k], v))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,D,G,N,ragged", [
    (480, 530, 8, 1, 4, True), (128, 530, 16, 4, 16, True), (128, 545, 24, 4, 16, False),
    (128, 530, 20, 4, 20, True), (240, 530, 10, 2, 40, True), (470, 500, 4, 1, 8, False)])
def test_scan_gradient_over_several_chunks_a_block(B, T, D, G, N, ragged, dtype):
    """Many rows: a block walks two or more chunks, its sums carried from one to the next,
    for state sizes whose dB and dC sums lie over used steps (up to 16) and beside them."""
    ln = 1
    while ln * 4 < N:
        ln *= 2
    wide = 64 // ln * (4 if ln <= 8 else 2 if ln == 16 else 1)
    parts, chunks, per = (D // G + wide - 1) // wide, (T + 31) // 32, 1
    while per < 8 and G * parts * B * (chunks // (2 * per)) >= 152 * 3 * 8:
        per *= 2
    assert per >= 2
    m, g = falcon(), _gen(B + T + D + N)
    d = dict(u=_draw(g, B, T, D, dtype=dtype), delta=(0.5 * _draw(g, B, T, D)).to(dtype),
             A=-torch.exp(_draw(g, D, N)), Bm=_draw(g, B, T, G, N, dtype=dtype),
             Cm=_draw(g, B, T, G, N, dtype=dtype), D=_draw(g, D), delta_bias=_draw(g, D) - 2.0,
             z=_draw(g, B, T, D, dtype=dtype), h0=_draw(g, B, D, N),
             lengths=_lengths(g, B, T) if ragged else None)
    dy, dh = _draw(g, B, T, D, dtype=dtype), _draw(g, B, D, N)
    want = vec.scan_gradients(**_wide(d), dy=dy.double(), dh_T=dh.double())
    if ragged:
        for b in range(B):
            n = int(d["lengths"][b])
            for t in (d["u"], d["delta"], d["Bm"], d["Cm"], d["z"], dy):
                t[b, n:] = float("nan")
    got = m.falcon_selective_scan_bwd(**d, dy=dy, dh_T=dh)
    tol = (T + 16) * 2.0 ** -21
    for k, v in want.items():
        half = dtype == BF16 and k in ("du", "ddelta", "dz", "dB", "dC")
        assert _rel(got[k], v) <= tol + (2.0 ** -8 if half else 0.0), (k, _rel(got[k], v))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("max_norm", [3.0, 1e9])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_clip_large_sets(dtype, max_norm, in_place):
    """Over 152 * 4 * 16384 elements (chunks of 16384, several a block) and over 40 MB (the
    first ones read as passing), with odd sizes and offsets."""
    m, g = falcon(), _gen(3)
    sizes = [9_000_001, 16384 * 700 + 1, 5, 1_234_567, 40_001, 16384, 3]
    assert sum(sizes) >= 152 * 4 * 16384 and sum(sizes) * (2 if dtype == BF16 else 4) > 40 << 20
    grads, outs = [], []
    for i, n in enumerate(sizes):
        grads.append((1e-3 * _draw(g, n + 3)).to(dtype)[i % 3:i % 3 + n])
        outs.append(torch.zeros(n + 3, dtype=dtype, device="cuda")[i % 2:i % 2 + n])
    n2 = sum(t.double().square().sum() for t in grads).sqrt()
    scale = min(1.0, max_norm / (float(n2) + 1e-6))
    want = [t.double() * scale for t in grads]
    norm = m.falcon_clip_grad_norm(grads, max_norm, out=None if in_place else outs)
    assert abs(float(norm) - float(n2)) <= 2.0 ** -18 * float(n2)
    tol = (2.0 ** -8 if dtype == BF16 else 0.0) + 2.0 ** -17
    for i, (o, w) in enumerate(zip(grads if in_place else outs, want)):
        assert bool(((o.double() - w).abs() <= tol * w.abs() + 1e-40).all()), i


@pytest.mark.parametrize("count", [64, 65])
def test_clip_of_dozens_of_tensors(count):
    m, g = falcon(), _gen(4)
    grads = [_draw(g, 1 + 37 * i % 501) for i in range(count)]
    n2 = float(sum(t.double().square().sum() for t in grads).sqrt())
    want = [t.double() * (0.5 / (n2 + 1e-6)) for t in grads]
    assert abs(float(m.falcon_clip_grad_norm(grads, 0.5)) - n2) <= 2.0 ** -18 * n2
    for t, w in zip(grads, want):
        assert _rel(t, w) <= 2.0 ** -18
