"""The linear attention block's kernels against the 64-bit forms, element by element.

Tolerances.  u = half a step of the activations' type (bf16 2^-8, fp32 2^-24).  Decay
attention: an output is a sum of terms of total size A, each rounded once to bf16 on
the tensor cores (a weighted q k, or a state), summed in fp32, and rounded once itself:
u (|o| + A) for bf16, and fp32's rounding of sums of m + T terms and of the weights
(exponents of up to 88 that are off by 2^-24 of themselves), 2^-23 (m + T + 256) A.  States
and their gradients are fp32 throughout: the second part alone, for sums over T tokens.
Gated norm: every step is fp32, and rounded once: u |y| and 2^-23 (D + 64) of the size of
what is summed (sums over rows: of B T terms too).
"""
import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def falcon():
    import delta_rule_attention_gb300 as falcon
    return falcon


@pytest.fixture(autouse=True)
def no_timeout(falcon):
    yield
    assert falcon.falcon_sync_check() == 0


def near(got, want, size, half, terms, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    tol = half * (want.abs() + size) * 1.01 + 2.0 ** -23 * terms * size + 1e-37
    off = (got - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol).max()))


def once(got, want, size, half, terms, what=""):
    """Rounded once: half a step of the value alone."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    tol = half * want.abs() * 1.01 + 2.0 ** -23 * terms * size + 1e-37
    off = (got - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol).max()))


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def decay_case(B, H, T, m, dv, dtype, seed=0, ends=True, lengths=None, rows=False):
    g = gen(seed)
    c = {}
    if rows:
        qkv = randn(g, B, T, H * (2 * m + dv), dtype=dtype)
        part = lambda a, w: qkv[..., a:a + H * w].unflatten(2, (H, w)).transpose(1, 2)  # noqa: E731
        c.update(q=part(0, m), k=part(H * m, m), v=part(2 * H * m, dv))
    else:
        c.update(q=randn(g, B, H, T, m, dtype=dtype), k=randn(g, B, H, T, m, dtype=dtype),
                 v=randn(g, B, H, T, dv, dtype=dtype))
    at = torch.arange(H, device="cuda") / max(H - 1, 1)
    c["log_decay"] = -torch.exp2(-0.5 - 11 * at)
    if ends:
        c["S0"] = randn(g, B, H, m, dv)
    if lengths is not None:
        c["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return c


SHAPES = [
    # B, H, T, m, dv
    (1, 1, 1, 64, 64), (2, 3, 17, 64, 64), (1, 2, 128, 64, 64), (2, 2, 129, 64, 64),
    (1, 2, 300, 128, 128), (2, 1, 257, 64, 128), (1, 3, 200, 128, 64), (2, 2, 70, 16, 32),
    (1, 2, 140, 40, 96), (1, 2, 65, 37, 5), (1, 1, 130, 1, 1), (2, 2, 64, 100, 128),
    (3, 5, 383, 48, 64),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,T,m,dv", SHAPES)
def test_decay_forward(falcon, B, H, T, m, dv, dtype):
    for ends, rows, lengths in ((True, False, None), (False, True, None),
                                (True, True, [T // 2 + 1, 0, T][:B])):
        c = decay_case(B, H, T, m, dv, dtype, seed=T + m, ends=ends, rows=rows, lengths=lengths)
        o, S = falcon.falcon_decay_attn_fwd(**c)
        want, want_S = ref.decay_forward(**c)
        size, size_S = ref.decay_forward_size(**c)
        near(o, want, size, HALF[dtype], m + T + 256, "o")
        near(S, want_S, size_S, 0.0, T + 256, "S")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,T,m,dv", SHAPES)
def test_decay_backward(falcon, B, H, T, m, dv, dtype):
    for ends, rows, lengths in ((True, False, None), (False, True, None),
                                (True, True, [T // 2 + 1, 0, T][:B])):
        c = decay_case(B, H, T, m, dv, dtype, seed=T + m, ends=ends, rows=rows, lengths=lengths)
        g = gen(T)
        c["dO"] = randn(g, B, H, T, dv, dtype=dtype)
        if ends:
            c["dS_T"] = randn(g, B, H, m, dv)
        got = falcon.falcon_decay_attn_bwd(**c)
        want, size = ref.decay_gradient(**c), ref.decay_gradient_size(**c)
        for name in ("dq", "dk", "dv"):
            near(got[name], want[name], size[name], HALF[dtype], m + dv + T + 256, name)
        near(got["dS0"], want["dS0"], size["dS0"], 0.0, T + 256, "dS0")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decay_extreme_rates(falcon, dtype):
    """No decay, a positive rate, one that forgets within a token, none left at all."""
    B, T, m = 1, 260, 64
    for scale in (1.0, -0.25):
        c = decay_case(B, 5, T, m, m, dtype, seed=3)
        c["log_decay"] = torch.tensor([0.0, 2.0, -30.0, -float("inf"), -3e38], device="cuda")
        c["scale"] = scale
        o, S = falcon.falcon_decay_attn_fwd(**c)
        want, want_S = ref.decay_forward(**c)
        size, size_S = ref.decay_forward_size(**c)
        near(o, want, size, HALF[dtype], m + T + 256, "o")
        near(S, want_S, size_S, 0.0, T + 256, "S")
        c["dO"], c["dS_T"] = randn(gen(4), B, 5, T, m, dtype=dtype), randn(gen(5), B, 5, m, m)
        got = falcon.falcon_decay_attn_bwd(**c)
        want, size = ref.decay_gradient(**c), ref.decay_gradient_size(**c)
        for name in ("dq", "dk", "dv"):
            near(got[name], want[name], size[name], HALF[dtype], 2 * m + T + 256, name)
        near(got["dS0"], want["dS0"], size["dS0"], 0.0, T + 256, "dS0")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decay_padding_is_not_read(falcon, dtype):
    B, H, T, m = 4, 2, 300, 64
    n = [0, 1, 130, 300]
    c = decay_case(B, H, T, m, m, dtype, seed=9, lengths=n)
    c["dO"] = randn(gen(1), B, H, T, m, dtype=dtype)
    for x in ("q", "k", "v", "dO"):
        for b in range(B):
            c[x][b, :, n[b]:] = float("nan")
    fwd = {x: t for x, t in c.items() if x != "dO"}
    o, S = falcon.falcon_decay_attn_fwd(**fwd)
    want, want_S = ref.decay_forward(**fwd)
    for b in range(B):
        assert (o[b, :, n[b]:] == 0).all()
    size, size_S = ref.decay_forward_size(**fwd)
    near(o, want, size, HALF[dtype], m + T + 256, "o")
    near(S, want_S, size_S, 0.0, T + 256, "S")
    got = falcon.falcon_decay_attn_bwd(**c)
    want, size = ref.decay_gradient(**c), ref.decay_gradient_size(**c)
    for name in ("dq", "dk", "dv"):
        near(got[name], want[name], size[name], HALF[dtype], 2 * m + T + 256, name)
        for b in range(B):
            assert (got[name][b, :, n[b]:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decay_layouts(falcon, dtype):
    """Broadcast heads and batches, single entries with any stride, unaligned rows, results
    in the middle of other tensors, the state in place."""
    B, H, T, m = 2, 3, 150, 64
    base = decay_case(B, H, T, m, m, dtype, seed=2)
    g = gen(7)
    one = randn(g, B, 1, T, m, dtype=dtype).expand(B, H, T, m)
    for name, t in (("k", one), ("v", randn(g, 1, 1, T, m, dtype=dtype).expand(B, H, T, m)),
                    ("q", randn(g, B, H, 1, m, dtype=dtype).expand(B, H, T, m)),
                    ("k", randn(g, B, H, T, m + 1, dtype=dtype)[..., 1:]),
                    ("v", randn(g, B, H, T + 1, 2 * m, dtype=dtype)[:, :, 1:, 8:8 + m])):
        c = {**base, name: t}
        want, want_S = ref.decay_forward(**c)
        size, size_S = ref.decay_forward_size(**c)
        room = torch.full((B, T + 2, H, m + 8), 7.0, dtype=dtype, device="cuda")
        out = room[:, 1:-1, :, 4:-4].transpose(1, 2)
        out8 = room[:, 1:-1, :, :m].transpose(1, 2)
        for to in (out, out8):
            room.fill_(7.0)
            S = c["S0"].clone()
            falcon.falcon_decay_attn_fwd(**{**c, "S0": S}, o=to, S_out=S)
            near(to, want, size, HALF[dtype], m + T + 256, name)
            near(S, want_S, size_S, 0.0, T + 256, "S")
            assert (room[:, 0] == 7).all() and (room[:, -1] == 7).all()
            to.fill_(7.0)
            assert (room == 7).all()


def test_decay_long(falcon):
    """Many runs a head against the same tokens in pieces, on both paths."""
    for dtype, m, T in ((BF16, 64, 20000), (BF16, 128, 9001), (F32, 64, 9001)):
        c = decay_case(1, 2, T, m, m, dtype, seed=5)
        o, S = falcon.falcon_decay_attn_fwd(**c)
        want, want_S = ref.decay_forward(**c)
        size, size_S = ref.decay_forward_size(**c)
        near(o, want, size, HALF[dtype], m + 1024, "o")
        near(S, want_S, size_S, 0.0, 1024, "S")
        cut = T // 3
        first = {**c, **{x: c[x][:, :, :cut] for x in "qkv"}}
        rest = {**c, **{x: c[x][:, :, cut:] for x in "qkv"}}
        o1, S1 = falcon.falcon_decay_attn_fwd(**first)
        o2, S2 = falcon.falcon_decay_attn_fwd(**{**rest, "S0": S1})
        near(torch.cat([o1, o2], 2), want, size, HALF[dtype], m + 1024, "pieces")
        near(S2, want_S, size_S, 0.0, 1024, "S of pieces")


def test_decay_of_no_token(falcon):
    c = decay_case(2, 3, 0, 64, 64, BF16)
    o, S = falcon.falcon_decay_attn_fwd(**c)
    assert o.shape == (2, 3, 0, 64) and torch.equal(S, c["S0"])
    g = falcon.falcon_decay_attn_bwd(**c, dO=o, dS_T=c["S0"] + 1)
    assert torch.equal(g["dS0"], c["S0"] + 1)
    S = falcon.falcon_decay_attn_fwd(**{**c, "S0": None})[1]
    assert (S == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,H,m,dv", [(1, 1, 1, 1), (3, 2, 64, 64), (5, 3, 128, 128), (2, 2, 37, 5),
                                      (4, 1, 128, 37), (3, 4, 16, 128), (2, 3, 100, 32)])
def test_decay_step(falcon, N, H, m, dv, dtype):
    g = gen(m + dv)
    pool = N + 3
    q, k = (randn(g, N, 2 * H, m, dtype=dtype)[:, ::2] for _ in range(2))
    v = randn(g, N, H, dv, dtype=dtype)
    log_decay = -torch.exp2(-torch.arange(H, device="cuda").float())
    S = randn(g, pool, H, m, dv)
    for slots, fresh in ((None, None), (list(range(pool))[::-1][:N], None),
                         ([pool - 1] + [-1] * (N - 1), [1] + [0] * (N - 1))):
        at = list(range(N)) if slots is None else slots
        P = S[:N].clone() if slots is None else S.clone()
        before = P.clone()
        out = falcon.falcon_decay_attn_step(
            q, k, v, log_decay, P,
            slots=None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda"),
            fresh=None if fresh is None else torch.tensor(fresh, dtype=torch.uint8, device="cuda"))
        touched = set()
        for i, s in enumerate(at):
            if not 0 <= s < P.shape[0]:
                assert (out[i] == 0).all()
                continue
            touched.add(s)
            S0 = before[s:s + 1] * (0 if fresh and fresh[i] else 1)
            one = dict(q=q[i:i + 1, :, None], k=k[i:i + 1, :, None], v=v[i:i + 1, :, None],
                       log_decay=log_decay, S0=S0)
            want, want_S = ref.decay_forward(**one)
            size, size_S = ref.decay_forward_size(**one)
            once(out[i:i + 1, :, None], want, size, HALF[dtype], m + 16, "o")
            once(P[s:s + 1], want_S, size_S, 0.0, 8, "S")
        for s in range(P.shape[0]):
            assert s in touched or torch.equal(P[s], before[s])


NORMS = [
    # B, H, T, m, heads first
    (2, 1, 3, 64, False), (2, 12, 5, 64, True), (1, 3, 7, 111, True), (2, 5, 4, 16, False),
    (1, 1, 9, 1, False), (1, 1, 4, 8192, False), (3, 1, 2, 777, False), (1, 2, 3, 4096, True),
    (2, 7, 3, 8, True), (1, 16, 2, 128, True), (4, 1, 33, 40, False), (1, 3, 2, 96, True),
    (1, 64, 2, 128, False), (1, 73, 3, 111, True), (2, 1, 40, 768, False), (1, 2, 5, 320, True),
]


def norm_case(B, H, T, m, heads, dtype, seed, z=True, scale=True, x=True, nxt=True, lengths=None,
              weight=True):
    g = gen(seed)
    D = H * m
    c = dict(eps=1e-5)
    if heads:
        c["h"] = randn(g, B, H, T, m, dtype=dtype)
    else:
        h = randn(g, B, T, D, dtype=dtype)
        c["h"] = h if H == 1 else h.unflatten(2, (H, m)).transpose(1, 2)
    if weight:
        c["weight"] = randn(g, D)
    if z:
        c["z"] = randn(g, B, T, 2 * D, dtype=dtype)[..., D:]
    if scale:
        c["scale"] = randn(g, D)
    if x:
        c["x"] = randn(g, B, T, D, dtype=dtype)
    if nxt:
        c["next_weight"] = randn(g, D)
    if lengths is not None:
        c["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return c


VARIANTS = [dict(), dict(z=False), dict(x=False, nxt=False, scale=False), dict(nxt=False),
            dict(weight=False, scale=False), dict(x=False)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,T,m,heads", NORMS)
def test_norm_forward(falcon, B, H, T, m, heads, dtype):
    for i, kw in enumerate(VARIANTS):
        lengths = [T - 1, 0, T + 5, -2][:B] if i % 2 else None
        gate = ("silu", "sigmoid", "identity")[i % 3]
        c = norm_case(B, H, T, m, heads, dtype, seed=i, lengths=lengths, **kw)
        out, nxt = falcon.falcon_gated_norm_fwd(gate=gate, **c)
        (y, u), (sy, su) = ref.norm_forward(gate=gate, **c)
        once(out, y, sy, HALF[dtype], H * m + 64, "out")
        assert (nxt is None) == (u is None)
        if u is not None:
            once(nxt, u, su, HALF[dtype], H * m + 64, "next")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,T,m,heads", NORMS)
def test_norm_backward(falcon, B, H, T, m, heads, dtype):
    D = H * m
    for i, kw in enumerate(VARIANTS):
        lengths = [T - 1, 0, T + 5, -2][:B] if i % 2 else None
        gate = ("silu", "sigmoid", "identity")[i % 3]
        c = norm_case(B, H, T, m, heads, dtype, seed=i, lengths=lengths, **kw)
        residual = c.pop("x", None) is not None
        g = gen(100 + i)
        dout = None if i == 5 else randn(g, B, T, D, dtype=dtype)
        more = dict(dnext=randn(g, B, T, D, dtype=dtype), out=randn(g, B, T, D, dtype=dtype)) \
            if "next_weight" in c else {}
        got = falcon.falcon_gated_norm_bwd(dout=dout, gate=gate, residual=residual, **more, **c)
        want, size = ref.norm_gradient(dout=dout, gate=gate, residual=residual,
                                       dnext=more.get("dnext"), out=more.get("out"), **c)
        assert {n for n, t in got.items() if t is not None} == set(want)
        for name, t in want.items():
            if name in ("dweight", "dscale", "dnext_weight"):
                once(got[name], t, size[name], 0.0, D + B * T + 64, name)
            else:
                once(got[name], t, size[name], HALF[dtype], D + 64, name)


def test_norm_before_the_first_block(falcon):
    g = gen(0)
    x, w = randn(g, 3, 5, 96, dtype=BF16), randn(g, 96)
    out, nxt = falcon.falcon_gated_norm_fwd(None, x=x, next_weight=w)
    assert out is x
    (_, u), (_, su) = ref.norm_forward(None, x=x, next_weight=w)
    once(nxt, u, su, HALF[BF16], 96 + 64, "next")
    d = randn(g, 3, 5, 96, dtype=BF16)
    got = falcon.falcon_gated_norm_bwd(None, None, dnext=d, out=x, next_weight=w)
    want, size = ref.norm_gradient(None, None, dnext=d, out=x, next_weight=w)
    once(got["dx"], want["dx"], size["dx"], HALF[BF16], 96 + 64, "dx")
    once(got["dnext_weight"], want["dnext_weight"], size["dnext_weight"], 0.0, 200, "dnext_weight")
    assert got["dh"] is None and got["dweight"] is None


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_in_place_and_padding(falcon, dtype):
    B, H, T, m = 3, 2, 9, 64
    n = [4, 0, 9]
    c = norm_case(B, H, T, m, True, dtype, seed=3, lengths=n)
    for b in range(B):
        c["h"][b, :, n[b]:] = float("nan")
        c["z"][b, n[b]:] = float("nan")
        c["x"][b, n[b]:] = float("inf")
    (y, u), (sy, su) = ref.norm_forward(**c)
    x = c["x"].clone()
    out, nxt = falcon.falcon_gated_norm_fwd(**{**c, "x": x}, out=x)
    assert out is x
    once(out, y, sy, HALF[dtype], H * m + 64, "out")
    once(nxt, u, su, HALF[dtype], H * m + 64, "next")
    d = randn(gen(1), B, T, H * m, dtype=dtype)
    for b in range(B):
        d[b, n[b]:] = float("nan")
        assert (out[b, n[b]:] == 0).all() and (nxt[b, n[b]:] == 0).all()
    c.pop("x")
    want, size = ref.norm_gradient(dout=d, dnext=d, out=y.to(dtype), **c)
    stored = y.to(dtype).cuda()
    dx = d.clone()
    got = falcon.falcon_gated_norm_bwd(dout=dx, dnext=d, out=stored, grads=dict(dx=dx), **c)
    assert got["dx"] is dx
    for name in ("dx", "dh", "dz"):
        once(got[name], want[name], size[name], HALF[dtype], H * m + 64, name)


def test_norm_of_zero_rows_and_of_no_row(falcon):
    z = torch.zeros(2, 3, 64, device="cuda", dtype=BF16)
    w = torch.ones(64, device="cuda")
    out, nxt = falcon.falcon_gated_norm_fwd(z, weight=w, x=z.clone(), next_weight=w)
    assert (out == 0).all() and (nxt == 0).all()
    g = falcon.falcon_gated_norm_bwd(z[:, :0], z[:, :0], weight=w)
    assert (g["dweight"] == 0).all() and g["dh"].shape == (2, 0, 64)


def test_norm_many_rows(falcon):
    """More rows than blocks take at once: the sums over a block's rows, and the blocks'."""
    for B, T, H, m, dtype in ((4, 5000, 1, 48, BF16), (1, 2500, 3, 37, F32)):
        c = norm_case(B, H, T, m, H > 1, dtype, seed=1)
        c.pop("x")
        g = gen(2)
        d, e, y = (randn(g, B, T, H * m, dtype=dtype) for _ in range(3))
        got = falcon.falcon_gated_norm_bwd(dout=d, dnext=e, out=y, **c)
        want, size = ref.norm_gradient(dout=d, dnext=e, out=y, **c)
        for name in ("dweight", "dscale", "dnext_weight"):
            # summed by thousands of threads: a tree of at most rows / 608 + 608 terms
            once(got[name], want[name], size[name], 0.0, H * m + 1024, name)
        once(got["dh"], want["dh"], size["dh"], HALF[dtype], H * m + 64, "dh")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 64, 65, 128, 129, 700])
def test_decay_gradient_of_the_state_in_place(falcon, T, dtype):
    """dS0 over dS_T, which the gradients of keys and values read."""
    c = decay_case(2, 3, T, 64, 64, dtype, seed=T, lengths=[T, T // 2])
    c["dO"], dS = randn(gen(1), 2, 3, T, 64, dtype=dtype), randn(gen(2), 2, 3, 64, 64)
    want = falcon.falcon_decay_attn_bwd(**c, dS_T=dS)
    held = dS.clone()
    got = falcon.falcon_decay_attn_bwd(**c, dS_T=held, grads=dict(dS0=held))
    assert got["dS0"] is held
    for name in ("dq", "dk", "dv", "dS0"):
        # the runs' states may be formed by another pass: the same sums in another order
        off = (got[name].double() - want[name].double()).abs()
        assert float(off.max()) <= 2 * HALF[dtype] * float(want[name].double().abs().max()) + 1e-4


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decay_mixed_layouts_in_the_gradient(falcon, dtype):
    """Results of which one lies where TMA cannot write or read: passes on both paths."""
    T, m = 300, 64
    c = decay_case(2, 2, T, m, m, dtype, seed=8)
    c["dO"], c["dS_T"] = randn(gen(1), 2, 2, T, m, dtype=dtype), randn(gen(2), 2, 2, m, m)
    want, size = ref.decay_gradient(**c), ref.decay_gradient_size(**c)
    odd = lambda: torch.empty(2, 2, T, m + 1, dtype=dtype, device="cuda")[..., 1:]  # noqa: E731
    for names in (("dq",), ("dk",), ("dv",), ("dq", "dv"), ("dk", "dv")):
        got = falcon.falcon_decay_attn_bwd(**c, grads={n: odd() for n in names})
        for name in ("dq", "dk", "dv"):
            near(got[name], want[name], size[name], HALF[dtype], 2 * m + T + 256, name)
        near(got["dS0"], want["dS0"], size["dS0"], 0.0, T + 256, "dS0")
