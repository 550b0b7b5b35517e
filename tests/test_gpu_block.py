"""The selective state space block's kernels against the float64 reference.

Tolerances, fixed before the first run: an output stored in bf16 is off by at
most 2^-8 of its value.  In fp32 a decay is off by 2^-22 (the exponential) and
2^-23 for each unit of its exponent, an addition by 2^-24; a state or adjoint
gathers at most one of each a token, so ||err|| / ||ref|| stays below
(T + 16) 2^-21.  A convolution of W <= 4 taps, its activation and the sums of its
gradients stay below 2^-18."""
import math

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def falcon():
    import delta_rule_attention_gb300 as m
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _draw(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def _tol(dtype, base):
    return base + (2.0 ** -8 if dtype == BF16 else 0.0)


def _same(got, want, dtype, base, name=""):
    assert got.dtype == dtype, name
    err = ref.rel(got, want)
    assert err <= _tol(dtype, base), (name, err)


# ------------------------------------------------------------ short convolution

CONV = 2.0 ** -18


def _conv_case(g, dtype, B, T, C, W, state, ragged):
    d = dict(x=_draw(g, B, T, C, dtype=dtype), weight=_draw(g, C, W), bias=_draw(g, C))
    d["state"] = _draw(g, B, W - 1, C, dtype=dtype) if state else None
    d["lengths"] = None
    if ragged:
        n = torch.randint(0, T + 1, (B,), generator=g)
        n[0] = 0
        n[-1] = T
        d["lengths"] = n.to(torch.int32)
    return d


def _ref_inputs(d):
    return {k: ref.f64(v) if isinstance(v, torch.Tensor) and v.is_floating_point() else v
            for k, v in d.items() if v is not None}


CONV_CASES = [(1, 1, 16, 4), (2, 2, 8, 3), (3, 37, 40, 4), (2, 65, 33, 2), (4, 130, 264, 4),
              (1, 515, 7, 3), (3, 16, 1030, 2), (2, 33, 8, 4)]


@pytest.mark.parametrize("activation", ["silu", "identity"])
@pytest.mark.parametrize("state,ragged", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("B,T,C,W", CONV_CASES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_forward_and_gradients(dtype, B, T, C, W, state, ragged, activation):
    g = _gen(B * 1000 + T * 10 + C + W)
    d = _conv_case(g, dtype, B, T, C, W, state, ragged)
    dy = _draw(g, B, T, C, dtype=dtype)
    dso = _draw(g, B, W - 1, C, dtype=dtype) if state else None
    c = _cuda(d)
    if ragged:  # what lies behind a row's length is never used
        for b in range(B):
            c["x"][b, int(d["lengths"][b]):] = float("nan")
    y, tail = falcon().falcon_short_conv_fwd(**c, activation=activation)
    got = falcon().falcon_short_conv_bwd(**c, dy=dy.cuda(),
                                         dstate_out=None if dso is None else dso.cuda(),
                                         activation=activation)
    r = _ref_inputs(d)
    want, wtail = ref.conv(**r, activation=activation)
    _same(y, want, dtype, CONV, "y")
    assert torch.equal(ref.f64(tail), wtail)
    cot = [ref.f64(dy), None if dso is None else ref.f64(dso)]
    if r.get("state") is None:
        r["state"] = torch.zeros(B, W - 1, C, dtype=torch.float64)
    grads = ref.gradients(lambda **k: ref.conv(**k, activation=activation), r, cot)
    _same(got["dx"], grads["x"], dtype, CONV, "dx")
    _same(got["dstate"], grads["state"], dtype, CONV, "dstate")
    _same(got["dweight"], grads["weight"], F32, CONV, "dweight")
    _same(got["dbias"], grads["bias"], F32, CONV, "dbias")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,m", [(3, 16), (2, 24), (5, 7)])
def test_conv_heads_from_projection_rows(dtype, H, m):
    B, T, W = 2, 41, 4
    g = _gen(H * m)
    rows = _draw(g, B, T, 3 * H * m, dtype=dtype).cuda()
    x = rows[..., H * m:2 * H * m].view(B, T, H, m).transpose(1, 2)  # strided heads
    w, bias, st = _draw(g, H * m, W), _draw(g, H * m), _draw(g, B, W - 1, H * m, dtype=dtype)
    dy = _draw(g, B, H, T, m, dtype=dtype)
    y, tail = falcon().falcon_short_conv_fwd(x, w.cuda(), bias=bias.cuda(), state=st.cuda())
    assert y.shape == (B, H, T, m) and y.is_contiguous()
    got = falcon().falcon_short_conv_bwd(x, w.cuda(), dy.cuda(), bias=bias.cuda(), state=st.cuda())
    flat = ref.f64(x).transpose(1, 2).reshape(B, T, H * m)
    r = dict(x=flat, weight=ref.f64(w), bias=ref.f64(bias), state=ref.f64(st))
    want, wtail = ref.conv(**r)
    _same(y.transpose(1, 2).reshape(B, T, H * m), want, dtype, CONV)
    assert torch.equal(ref.f64(tail), wtail)
    grads = ref.gradients(ref.conv, r, [ref.f64(dy).transpose(1, 2).reshape(B, T, H * m), None])
    _same(got["dx"].transpose(1, 2).reshape(B, T, H * m), grads["x"], dtype, CONV)
    _same(got["dweight"], grads["weight"], F32, CONV)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_unaligned_views(dtype):
    g = _gen(5)
    rows = _draw(g, 2, 19, 50, dtype=dtype).cuda()
    x = rows[:, 1:, 1:41]  # an odd first channel, an odd first row
    w = _draw(g, 40, 4)
    y, tail = falcon().falcon_short_conv_fwd(x, w.cuda())
    want, wtail = ref.conv(ref.f64(x), ref.f64(w))
    _same(y, want, dtype, CONV)
    assert torch.equal(ref.f64(tail), wtail)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_of_no_token_passes_the_state(dtype):
    g = _gen(6)
    x = torch.empty(2, 0, 24, dtype=dtype, device="cuda")
    w, st = _draw(g, 24, 4).cuda(), _draw(g, 2, 3, 24, dtype=dtype).cuda()
    y, tail = falcon().falcon_short_conv_fwd(x, w, state=st)
    assert y.shape == x.shape and torch.equal(tail, st)
    got = falcon().falcon_short_conv_bwd(x, w, x, state=st, dstate_out=st)
    assert torch.equal(got["dstate"], st)
    assert not got["dweight"].any() and not got["dbias"].any()


@pytest.mark.parametrize("activation", ["silu", "identity"])
@pytest.mark.parametrize("N,C,W", [(1, 16, 4), (5, 33, 3), (17, 264, 2), (300, 8, 4)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_step(dtype, N, C, W, activation):
    g = _gen(N + C + W)
    pool = N + 3
    x, w, bias = _draw(g, N, C, dtype=dtype), _draw(g, C, W), _draw(g, C)
    st = _draw(g, pool, W - 1, C, dtype=dtype)
    slots = torch.randperm(pool, generator=g)[:N].to(torch.int32)
    fresh = (torch.rand(N, generator=g) < 0.3).to(torch.uint8)
    if N > 4:
        slots[1], slots[2] = -1, pool  # no such state
    sc = st.cuda()
    y = falcon().falcon_short_conv_step(x.cuda(), w.cuda(), sc, bias=bias.cuda(),
                                        slots=slots.cuda(), fresh=fresh.cuda(),
                                        activation=activation)
    want, pool_want = torch.zeros(N, C, dtype=torch.float64), st.clone()
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pool:
            before = torch.zeros_like(st[s]) if fresh[i] else st[s]
            o, tail = ref.conv(ref.f64(x[i])[None, None], ref.f64(w), ref.f64(bias),
                               ref.f64(before)[None], activation=activation)
            want[i], pool_want[s] = o[0, 0], tail[0].to(dtype)
    _same(y, want, dtype, CONV)
    assert torch.equal(sc.cpu(), pool_want)


# --------------------------------------------------------------- selective scan

def _scan_case(g, dtype, B, T, D, G, N, gate=True, state=False, ragged=False, full=True):
    d = dict(u=_draw(g, B, T, D, dtype=dtype), delta=_draw(g, B, T, D, dtype=dtype, scale=0.5),
             A=-torch.exp(_draw(g, D, N)), Bm=_draw(g, B, T, G, N, dtype=dtype),
             Cm=_draw(g, B, T, G, N, dtype=dtype))
    d["D"] = _draw(g, D) if full else None
    d["delta_bias"] = _draw(g, D) - 2.0 if full else None
    d["z"] = _draw(g, B, T, D, dtype=dtype) if gate else None
    d["h0"] = _draw(g, B, D, N) if state else None
    d["lengths"] = None
    if ragged:
        n = torch.randint(0, T + 1, (B,), generator=g)
        n[0] = 0
        n[-1] = T
        d["lengths"] = n.to(torch.int32)
    return d


def _scan_check(d, dtype, softplus=True, poison=False):
    B, T, D = d["u"].shape
    N = d["A"].shape[1]
    g = _gen(99)
    dy = _draw(g, B, T, D, dtype=dtype)
    dh = _draw(g, B, D, N) if d["h0"] is not None else None
    c, dyc = _cuda(d), dy.cuda()
    if poison:
        for b in range(B):
            n = int(d["lengths"][b])
            for k in ("u", "delta", "Bm", "Cm", "z"):
                if c[k] is not None:
                    c[k][b, n:] = float("nan")
            dyc[b, n:] = float("inf")
    tol = (T + 16) * 2.0 ** -21
    y, h = falcon().falcon_selective_scan_fwd(**c, softplus=softplus)
    got = falcon().falcon_selective_scan_bwd(**c, dy=dyc, dh_T=None if dh is None else dh.cuda(),
                                             softplus=softplus)
    r = _ref_inputs(d)
    want, hw = ref.scan(**r, softplus=softplus)
    _same(y, want, dtype, tol, "y")
    _same(h, hw, F32, tol, "h")
    r.setdefault("h0", torch.zeros(B, D, N, dtype=torch.float64))
    grads = ref.gradients(lambda **k: ref.scan(**k, softplus=softplus), r,
                          [ref.f64(dy), ref.f64(dh)])
    for mine, theirs, dt in (("du", "u", dtype), ("ddelta", "delta", dtype), ("dz", "z", dtype),
                             ("dB", "Bm", dtype), ("dC", "Cm", dtype), ("dA", "A", F32),
                             ("dD", "D", F32), ("ddelta_bias", "delta_bias", F32),
                             ("dh0", "h0", F32)):
        if theirs in grads:
            _same(got[mine], grads[theirs], dt, tol, mine)
        else:
            assert got[mine] is None, mine


@pytest.mark.parametrize("N", [1, 3, 4, 5, 8, 16, 24, 33, 64, 100, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_state_sizes(dtype, N):
    g = _gen(N)
    _scan_check(_scan_case(g, dtype, 2, 21, 24, 2, N, state=True), dtype)


@pytest.mark.parametrize("B,D,G", [(1, 8, 1), (3, 1, 1), (2, 40, 4), (1, 77, 7), (2, 264, 1),
                                   (1, 130, 2)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_channels_and_groups(dtype, B, D, G):
    g = _gen(D)
    _scan_check(_scan_case(g, dtype, B, 19, D, G, 16), dtype)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 127, 130, 300])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_lengths(dtype, T):
    g = _gen(T)
    _scan_check(_scan_case(g, dtype, 2, T, 16, 1, 16, state=T % 2 == 1), dtype)


@pytest.mark.parametrize("T,D,N,ragged", [(1301, 16, 16, True), (1100, 40, 8, False),
                                          (600, 8, 33, True), (1030, 6, 1, True)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_split_over_many_segments(dtype, T, D, N, ragged):
    g = _gen(T)
    _scan_check(_scan_case(g, dtype, 2, T, D, 1, N, state=True, ragged=ragged), dtype,
                poison=ragged)


@pytest.mark.parametrize("T,N,G", [(1, 16, 1), (9, 16, 2), (40, 16, 1), (130, 8, 4), (67, 40, 1),
                                   (257, 16, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_ragged_rows_ignore_what_lies_behind(dtype, T, N, G):
    g = _gen(T + N)
    _scan_check(_scan_case(g, dtype, 4, T, 24, G, N, state=True, ragged=True), dtype, poison=True)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("gate,full", [(False, False), (True, False), (False, True)])
def test_scan_without_its_options(gate, full, softplus):
    g = _gen(7)
    d = _scan_case(g, F32, 2, 20, 16, 1, 16, gate=gate, full=full)
    if not softplus:
        d["delta"] = d["delta"].abs() * 0.1  # steps are used as they are: keep them positive
        if full:
            d["delta_bias"] = d["delta_bias"].abs() * 0.1
    _scan_check(d, F32, softplus=softplus)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_strided_views(dtype):
    B, T, D, G, N = 2, 35, 48, 2, 16
    g = _gen(8)
    d = _scan_case(g, dtype, B, T, D, G, N)
    uz = torch.cat([d["u"], d["z"]], -1).cuda()
    pad = _draw(g, B, T, 3, dtype=dtype)  # an odd offset: no vector access fits
    bc = torch.cat([pad, d["Bm"].flatten(2), d["Cm"].flatten(2)], -1).cuda()
    c = _cuda(d)
    views = dict(c, u=uz[..., :D], z=uz[..., D:], Bm=bc[..., 3:3 + G * N].view(B, T, G, N),
                 Cm=bc[..., 3 + G * N:].view(B, T, G, N))
    y0, h0 = falcon().falcon_selective_scan_fwd(**c)
    y1, h1 = falcon().falcon_selective_scan_fwd(**views)
    tol = (T + 16) * 2.0 ** -21
    assert ref.rel(y1, ref.f64(y0)) <= _tol(dtype, tol) and ref.rel(h1, ref.f64(h0)) <= tol
    dy = _draw(g, B, T, D, dtype=dtype).cuda()
    a, b = (falcon().falcon_selective_scan_bwd(**v, dy=dy) for v in (c, views))
    for k in a:
        assert ref.rel(b[k], ref.f64(a[k])) <= _tol(dtype, tol), k


def test_scan_of_no_token_passes_the_state():
    g = _gen(9)
    d = _cuda(_scan_case(g, F32, 2, 0, 16, 1, 16, state=True))
    y, h = falcon().falcon_selective_scan_fwd(**d)
    assert y.shape == (2, 0, 16) and torch.equal(h, d["h0"])
    dh = _draw(g, 2, 16, 16).cuda()
    got = falcon().falcon_selective_scan_bwd(**d, dy=d["u"], dh_T=dh)
    assert torch.equal(got["dh0"], dh)
    assert not got["dA"].any() and not got["dD"].any() and not got["ddelta_bias"].any()


def test_scan_states_may_be_updated_in_place():
    g = _gen(10)
    d = _cuda(_scan_case(g, F32, 2, 50, 40, 1, 16, state=True))
    y, h = falcon().falcon_selective_scan_fwd(**d)
    mine = d["h0"].clone()
    y2, h2 = falcon().falcon_selective_scan_fwd(**{**d, "h0": mine}, h_out=mine)
    assert torch.equal(y, y2) and torch.equal(h, h2) and h2 is mine


def test_scan_extreme_steps():
    """Steps of zero leave the state, large ones erase it, and neither is NaN."""
    g = _gen(11)
    d = _scan_case(g, F32, 1, 6, 8, 1, 16, state=True)
    d["delta"][0, 0] = -float("inf")
    d["delta"][0, 1] = -200.0
    d["delta"][0, 2] = 300.0
    d["delta"][0, 3] = 25.0
    y, h = falcon().falcon_selective_scan_fwd(**_cuda(d))
    want, hw = ref.scan(**_ref_inputs(d))
    tol = (6 + 16) * 2.0 ** -21 + 300 * 2.0 ** -23
    _same(y, want, F32, tol)
    _same(h, hw, F32, tol)


def test_scan_gradient_against_differences():
    """The kernel's own forward, moved along a direction in every input."""
    g = _gen(12)
    d = _cuda(_scan_case(g, F32, 2, 33, 24, 2, 16, state=True))
    dy, dh = _draw(g, 2, 33, 24).cuda(), _draw(g, 2, 24, 16).cuda()
    grads = falcon().falcon_selective_scan_bwd(**d, dy=dy, dh_T=dh)
    names = dict(u="du", delta="ddelta", A="dA", Bm="dB", Cm="dC", D="dD", z="dz",
                 delta_bias="ddelta_bias", h0="dh0")

    def total(inputs):
        y, h = falcon().falcon_selective_scan_fwd(**inputs)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())

    for k, name in names.items():
        v = grads[name] / grads[name].norm()  # the steepest direction
        step = 2.0 ** -7
        num = (total({**d, k: d[k] + step * v}) - total({**d, k: d[k] - step * v})) / (2 * step)
        # third-order term ~ step^2 = 6e-5 of the derivative, rounding 1e-6 / step
        assert abs(num - float(grads[name].norm())) <= 2e-3 * float(grads[name].norm()), k


@pytest.mark.parametrize("N,D,G,S", [(1, 16, 1, 16), (3, 33, 3, 5), (40, 24, 2, 16), (9, 8, 1, 128),
                                     (6, 40, 1, 1), (5, 264, 1, 24)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_step(dtype, N, D, G, S):
    g = _gen(N + D + S)
    d = _scan_case(g, dtype, N, 1, D, G, S)
    pool = N + 2
    h = _draw(g, pool, D, S)
    slots = torch.randperm(pool, generator=g)[:N].to(torch.int32)
    fresh = (torch.rand(N, generator=g) < 0.3).to(torch.uint8)
    if N > 4:
        slots[1], slots[2] = -7, pool + 1  # no such state
    hc = h.cuda()
    one = {k: d[k][:, 0].cuda() for k in ("u", "delta", "Bm", "Cm", "z")}
    y = falcon().falcon_selective_scan_step(
        one["u"], one["delta"], d["A"].cuda(), one["Bm"], one["Cm"], hc, D=d["D"].cuda(),
        z=one["z"], delta_bias=d["delta_bias"].cuda(), slots=slots.cuda(), fresh=fresh.cuda())
    r = _ref_inputs(d)
    want, hw = torch.zeros(N, D, dtype=torch.float64), ref.f64(h)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pool:
            before = torch.zeros_like(hw[s]) if fresh[i] else hw[s].clone()
            row = {k: (v[i:i + 1] if k in one else v) for k, v in r.items()}
            o, hn = ref.scan(**row, h0=before[None])
            want[i], hw[s] = o[0, 0], hn[0]
    tol = 17 * 2.0 ** -21
    _same(y, want, dtype, tol)
    _same(hc, hw, F32, tol)


# --------------------------------------------------------------------- together

def test_prompt_then_tokens_is_the_longer_prompt():
    g = _gen(13)
    B, T, D, N, W, dtype = 3, 20, 32, 16, 4, BF16
    d = _cuda(_scan_case(g, dtype, B, T, D, 1, N))
    w, bias = _draw(g, D, W).cuda(), _draw(g, D).cuda()
    m = falcon()
    xs, tail = m.falcon_short_conv_fwd(d["u"], w, bias=bias)
    y, h = m.falcon_selective_scan_fwd(**{**d, "u": xs})
    cut = 13
    first = {k: v[:, :cut] if k in ("u", "delta", "Bm", "Cm", "z") else v for k, v in d.items()}
    x1, st = m.falcon_short_conv_fwd(first["u"], w, bias=bias)
    y1, h1 = m.falcon_selective_scan_fwd(**{**first, "u": x1})
    rows = [y1]
    for t in range(cut, T):
        xt = m.falcon_short_conv_step(d["u"][:, t], w, st, bias=bias)
        rows.append(m.falcon_selective_scan_step(
            xt, d["delta"][:, t], d["A"], d["Bm"][:, t], d["Cm"][:, t], h1, D=d["D"],
            z=d["z"][:, t], delta_bias=d["delta_bias"])[:, None])
    assert torch.equal(st, tail)
    assert ref.rel(h1, ref.f64(h)) <= (T + 16) * 2.0 ** -21
    assert ref.rel(torch.cat(rows, 1), ref.f64(y)) <= 2.0 ** -7  # two roundings


def test_calls_run_on_the_callers_stream_and_in_graphs():
    g = _gen(14)
    m = falcon()
    d = _cuda(_scan_case(g, BF16, 2, 70, 64, 1, 16))
    w = _draw(g, 64, 4).cuda()
    dy = _draw(g, 2, 70, 64, dtype=BF16).cuda()
    outs = [torch.empty_like(dy) for _ in range(2)]

    def block():
        xs, _ = m.falcon_short_conv_fwd(d["u"], w)
        y, _ = m.falcon_selective_scan_fwd(**{**d, "u": xs})
        gr = m.falcon_selective_scan_bwd(**{**d, "u": xs}, dy=dy)
        cv = m.falcon_short_conv_bwd(d["u"], w, gr["du"])
        norm = m.falcon_clip_grad_norm([gr["dA"], cv["dweight"], cv["dx"]], 0.5)
        return y, cv["dx"], cv["dweight"], gr["dA"], norm

    want = [t.clone() for t in block()]
    again = block()
    assert all(torch.equal(a, b) for a, b in zip(want, again)), "results vary between runs"
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = block()
    for t in kept:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept))
    del outs


def test_calls_on_a_given_stream_keep_their_memory():
    """A call on another stream than the current one: what it allocates is not handed
    out again before the call is done with it."""
    g = _gen(17)
    m = falcon()
    d = _cuda(_scan_case(g, BF16, 2, 600, 256, 1, 16))
    dy = _draw(g, 2, 600, 256, dtype=BF16).cuda()
    w = _draw(g, 256, 4).cuda()
    want = m.falcon_selective_scan_bwd(**d, dy=dy)
    cw = m.falcon_short_conv_bwd(d["u"], w, dy)
    n0 = m.falcon_clip_grad_norm([want["dA"]], 1e9)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = m.falcon_selective_scan_bwd(**d, dy=dy, stream=side)
        cg = m.falcon_short_conv_bwd(d["u"], w, dy, stream=side)
        n1 = m.falcon_clip_grad_norm([want["dA"]], 1e9, stream=side)
        # the current stream writes over whatever the allocator holds free
        for _ in range(8):
            torch.full((1 << 22,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
        assert all(torch.equal(cg[k], cw[k]) for k in cw)
        assert float(n0) == float(n1)


def test_no_row_at_all():
    m = falcon()
    x = torch.empty(0, 5, 16, device="cuda")
    w = torch.ones(16, 4, device="cuda")
    y, tail = m.falcon_short_conv_fwd(x, w)
    assert y.shape == x.shape and tail.shape == (0, 3, 16)
    got = m.falcon_short_conv_bwd(x, w, x)
    assert not got["dweight"].any() and not got["dbias"].any()
    A, bc = -torch.ones(16, 8, device="cuda"), torch.empty(0, 5, 1, 8, device="cuda")
    y, h = m.falcon_selective_scan_fwd(x, x, A, bc, bc)
    assert h.shape == (0, 16, 8)
    got = m.falcon_selective_scan_bwd(x, x, A, bc, bc, x, D=torch.ones(16, device="cuda"))
    assert not got["dA"].any() and not got["dD"].any()
    one = torch.empty(0, 16, device="cuda")
    assert m.falcon_short_conv_step(one, w, torch.empty(0, 3, 16, device="cuda")).shape == (0, 16)


# ------------------------------------------------------------------------- clip

def _clip_ref(grads, max_norm, eps=1e-6):
    n = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))
    return n, min(1.0, max_norm / (n + eps))


@pytest.mark.parametrize("max_norm", [0.0, 0.37, 1e9])
@pytest.mark.parametrize("in_place", [True, False])
def test_clip_mixed_sizes_and_types(max_norm, in_place):
    g = _gen(15)
    sizes = [1, 3, 0, 8, 17, 255, 4096, 16384, 16385, 50001, 7]
    flat = _draw(g, 200000).cuda()
    flat16 = _draw(g, 200000, dtype=BF16).cuda()
    grads, at = [], 1
    for i, n in enumerate(sizes):  # views at odd offsets, both types
        src = flat if i % 2 else flat16
        grads.append(src[at:at + n])
        at += n
    n, scale = _clip_ref([t.cpu() for t in grads], max_norm)
    want = [t.double() * scale for t in grads]
    keep = [t.clone() for t in grads]
    out = None if in_place else [torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
                                 for t in grads]
    norm = falcon().falcon_clip_grad_norm(grads, max_norm, out=out)
    # squares, sums and the scale: a few roundings each, sums in float64 across threads
    assert abs(float(norm) - n) <= 2.0 ** -18 * n
    for i, (o, w_) in enumerate(zip(grads if in_place else out, want)):
        off = (o.double() - w_).abs()
        tol = (2.0 ** -8 if o.dtype == BF16 else 0.0) + 2.0 ** -17
        assert bool((off <= tol * w_.abs() + 1e-45).all()), i
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(keep, grads))
    if in_place and max_norm == 1e9:
        assert all(torch.equal(a, b) for a, b in zip(keep, grads))


@pytest.mark.parametrize("count", [1, 511, 512, 513, 1500])
def test_clip_many_tensors(count):
    g = _gen(16)
    flat = _draw(g, count * 13).cuda()
    grads = [flat[i * 13:i * 13 + 1 + i % 13] for i in range(count)]
    want = [t.clone() for t in grads]
    n, scale = _clip_ref([t.cpu() for t in grads], 1.0)
    norm = falcon().falcon_clip_grad_norm(grads, 1.0)
    assert abs(float(norm) - n) <= 2.0 ** -18 * n
    got, ref_ = torch.cat(grads), torch.cat(want)
    assert ref.rel(got, ref.f64(ref_) * scale) <= 2.0 ** -18


def test_clip_special_values():
    m = falcon()
    one = lambda *v: torch.tensor(v, device="cuda")  # noqa: E731
    a = one(0.0, 0.0)
    assert float(m.falcon_clip_grad_norm([a], 1.0)) == 0.0 and not a.any()
    a, b = one(1.0, float("nan")), one(2.0)
    assert math.isnan(float(m.falcon_clip_grad_norm([a, b], 1.0)))
    assert bool(a.isnan().all()) and bool(b.isnan().all())
    a, b = one(1.0, float("inf")), one(2.0)
    assert math.isinf(float(m.falcon_clip_grad_norm([a, b], 1.0)))
    assert a[0] == 0 and a[1].isnan() and b[0] == 0
    e = torch.empty(0, device="cuda")
    assert float(m.falcon_clip_grad_norm([e], 1.0)) == 0.0
