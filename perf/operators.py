"""The operators of a selective state space block, as cases to time and to check.

Three operators, each in the forms that a program needs:

  short convolution   y_t = act(b + sum_j w_j x_{t-W+1+j}), one filter a channel,
                      over prompts, its gradient, and one token of many sequences;
  selective scan      h_t = exp(D_t A) h_{t-1} + D_t B_t u_t, y_t = <C_t, h_t> + D u_t,
                      gated by silu(z), over prompts, its gradient, and one token;
  gradient clipping   the norm over all gradients of a step, and their scaling.

`own` False computes each in plain torch operations, `own` True through the
package's entry points.  `exact` computes the same from the definitions in
64 bits, token by token.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_CLIP_EPS = 1e-6


def listed():
    return [
        # The convolution over the keys of a language-model layer: read from the
        # projection's [B, T, H m] rows, written head by head for the attention.
        dict(name="conv prompt heads", op="conv_fwd", dtype="bf16", B=8, H=12, T=2048, m=64,
             W=4, act="silu", state=False, ragged=False),
        # Continued prompts of uneven lengths with an odd channel count.
        dict(name="conv ragged odd", op="conv_fwd", dtype="f32", B=5, H=1, T=777, m=331, W=3,
             act="identity", state=True, ragged=True),
        # The training step's gradient of the block's convolution.
        dict(name="conv backward", op="conv_bwd", dtype="bf16", B=8, H=1, T=2048, m=2048, W=4,
             act="silu", state=False, ragged=False),
        # One token for a serving batch, states in a pool of slots: latency.
        dict(name="conv step", op="conv_step", dtype="bf16", N=256, C=2048, W=4, act="silu"),
        # A batch of training sequences or prompts.
        dict(name="scan prompt", op="scan_fwd", dtype="bf16", B=8, T=2048, D=2048, G=1, N=16,
             gate=True, state=False, ragged=False),
        # One long document: few channels, many tokens.
        dict(name="scan long", op="scan_fwd", dtype="bf16", B=1, T=65536, D=2048, G=1, N=16,
             gate=True, state=False, ragged=False),
        # A few short continued prompts: latency.
        dict(name="scan short ragged", op="scan_fwd", dtype="f32", B=3, T=37, D=96, G=1, N=16,
             gate=True, state=True, ragged=True),
        # The training step's gradient of the scan.
        dict(name="scan backward", op="scan_bwd", dtype="bf16", B=8, T=2048, D=2048, G=1, N=16,
             gate=True, state=False, ragged=False),
        # Gradients through carried states, shared groups, an odd state size, no gate.
        dict(name="scan backward groups", op="scan_bwd", dtype="f32", B=2, T=517, D=200, G=4,
             N=24, gate=False, state=True, ragged=True),
        # One token for a large serving batch, states in a pool of slots.
        dict(name="scan step", op="scan_step", dtype="bf16", N=1024, D=2048, G=1, S=16,
             gate=True),
        # All gradients of a model of about 130 M parameters.
        dict(name="clip model", op="clip", dtype="bf16", layers=12, width=768, rows=32000,
             odd=False, clips=True),
        # A small model's odd-sized gradients, packed one behind the other.
        dict(name="clip small odd", op="clip", dtype="f32", layers=40, width=37, rows=411,
             odd=True, clips=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd",
                     "scan_bwd", "scan_step", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv_fwd", "conv_bwd"):
        H = rng.choice([1, 1, 12, 16])
        m = _log_int(rng, 16, 2048) if H == 1 else rng.choice([16, 32, 64, 128])
        if H == 1 and rng.random() < 0.6:
            m = (m + 7) // 8 * 8
        T = _log_int(rng, 1, 16384)
        B = min(_log_int(rng, 1, 32), max(1, (1 << 24) // (T * H * m)))
        return dict(op=op, dtype=dtype, B=B, H=H, T=T, m=m, W=rng.choice([2, 3, 4, 4]),
                    act=rng.choice(["silu", "silu", "identity"]), state=rng.random() < 0.5,
                    ragged=rng.random() < 0.4)
    if op == "conv_step":
        return dict(op=op, dtype=dtype, N=_log_int(rng, 1, 2048), C=_log_int(rng, 16, 2048),
                    W=rng.choice([2, 3, 4, 4]), act=rng.choice(["silu", "identity"]))
    if op in ("scan_fwd", "scan_bwd"):
        G = rng.choice([1, 1, 2, 4])
        D = G * _log_int(rng, 8, 2048 // G)
        if rng.random() < 0.6:
            D = (D + 8 * G - 1) // (8 * G) * (8 * G)
        N = rng.choice([4, 8, 16, 16, 16, 24, 32, 64, 5])
        T = _log_int(rng, 1, 16384)
        most = (1 << 28) // (D * N)  # tokens
        T = min(T, most)
        B = min(_log_int(rng, 1, 32), max(1, most // T))
        return dict(op=op, dtype=dtype, B=B, T=T, D=D, G=G, N=N, gate=rng.random() < 0.7,
                    state=rng.random() < 0.5, ragged=rng.random() < 0.4)
    if op == "scan_step":
        G = rng.choice([1, 1, 2])
        return dict(op=op, dtype=dtype, N=_log_int(rng, 1, 1024), D=G * _log_int(rng, 8, 2048 // G),
                    G=G, S=rng.choice([4, 8, 16, 16]), gate=rng.random() < 0.7)
    return dict(op=op, dtype=dtype, layers=rng.randint(1, 12), width=_log_int(rng, 16, 768),
                rows=_log_int(rng, 16, 32000), odd=rng.random() < 0.5, clips=rng.random() < 0.7)


# --------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _lengths(g, case):
    """Uneven lengths, 0 and T among them where there are rows enough."""
    n = torch.randint(0, case["T"] + 1, (case["B"],), generator=g, device="cuda")
    n[0] = case["T"]
    if case["B"] > 2:
        n[1] = 0
    return n.to(torch.int32)


def _slots(g, n, pool):
    return torch.randperm(pool, generator=g, device="cuda")[:n].to(torch.int32)


def _prepare_conv(case, g, dt):
    B, H, T, m, W = (case[k] for k in ("B", "H", "T", "m", "W"))
    s = dict(case=case)
    # the projection's rows [B, T, H m], seen head by head
    x = _randn(g, B, T, H * m, dtype=dt)
    s["x"] = x if H == 1 else x.view(B, T, H, m).transpose(1, 2)
    s["weight"] = _randn(g, H * m, W) * W ** -0.5
    s["bias"] = _randn(g, H * m) * 0.1
    s["state"] = _randn(g, B, W - 1, H * m, dtype=dt) if case["state"] else None
    s["lengths"] = _lengths(g, case) if case["ragged"] else None
    if case["op"] == "conv_bwd":
        s["dy"] = _randn(g, *s["x"].shape, dtype=dt)
        s["dstate_out"] = _randn(g, B, W - 1, H * m, dtype=dt) if case["state"] else None
    return s


def _prepare_scan(case, g, dt):
    step = case["op"] == "scan_step"
    lead = (case["N"],) if step else (case["B"], case["T"])
    D, G, N = case["D"], case["G"], case["S"] if step else case["N"]
    s = dict(case=case)
    # u beside the gate in one projection's rows, B and C beside the rank of
    # delta's projection: views with the rows' strides
    uz = _randn(g, *lead, 2 * D, dtype=dt)
    s["u"] = uz[..., :D]
    s["z"] = uz[..., D:] if case["gate"] else None
    rank = (D // 16 + 7) // 8 * 8
    bc = _randn(g, *lead, rank + 2 * G * N, dtype=dt)
    s["Bm"] = bc[..., rank:rank + G * N].view(*lead, G, N)
    s["Cm"] = bc[..., rank + G * N:].view(*lead, G, N)
    s["delta"] = (_randn(g, *lead, D) * 0.5).to(dt)
    # A starts at -1 .. -N, the steps spread over 0.001 .. 0.1
    n = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
    s["A"] = -n * torch.exp(0.1 * _randn(g, D, N))
    dt0 = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    s["delta_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    s["D"] = 1.0 + 0.1 * _randn(g, D)
    if step:
        pool = case["N"] + case["N"] // 16 + 1
        s["h"] = _randn(g, pool, D, N)
        s["slots"] = _slots(g, case["N"], pool)
        return s
    s["h0"] = _randn(g, case["B"], D, N) if case["state"] else None
    s["lengths"] = _lengths(g, case) if case["ragged"] else None
    if case["op"] == "scan_bwd":
        s["dy"] = _randn(g, *lead, D, dtype=dt)
        s["dh_T"] = _randn(g, case["B"], D, N) if case["state"] else None
    return s


def _clip_shapes(case):
    w, odd = case["width"], case["odd"]
    layer = [(w, 3 * w), (w, w + 1 if odd else w), (w, 5 * w // 2), (5 * w // 2, w), (w,)]
    return [(case["rows"], w)] + layer * case["layers"]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dt = _DTYPES[case["dtype"]]
    if op in ("conv_fwd", "conv_bwd"):
        return _prepare_conv(case, g, dt)
    if op == "conv_step":
        N, C, W = case["N"], case["C"], case["W"]
        pool = N + N // 16 + 1
        return dict(case=case, x=_randn(g, N, C, dtype=dt), weight=_randn(g, C, W) * W ** -0.5,
                    bias=_randn(g, C) * 0.1, state=_randn(g, pool, W - 1, C, dtype=dt),
                    slots=_slots(g, N, pool))
    if op in ("scan_fwd", "scan_bwd", "scan_step"):
        return _prepare_scan(case, g, dt)
    # gradients of a step, most of them small, and where the clipped ones go
    shapes = _clip_shapes(case)
    sizes = [math.prod(sh) for sh in shapes]
    # odd: packed one behind the other; otherwise each starts on 256 bytes
    up = 1 if case["odd"] else 128
    at = [sum((n + up - 1) // up * up for n in sizes[:i]) for i in range(len(sizes) + 1)]
    flat = (_randn(g, at[-1]) * 1e-3).to(dt)
    out = torch.zeros(at[-1], dtype=dt, device="cuda")
    cut = lambda t: [t[a:a + n].view(sh) for a, n, sh in zip(at, sizes, shapes)]  # noqa: E731
    big = 1e-3 * math.sqrt(sum(sizes))
    return dict(case=case, grads=cut(flat), out=out, outs=cut(out),
                max_norm=0.25 * big if case["clips"] else 4.0 * big)


# ---------------------------------------------------------------- plain forms

def _rows(x):
    """[B, H, T, m] as [B, T, H m]."""
    return x if x.dim() == 3 else x.transpose(1, 2).flatten(2)


def _heads(y, like):
    """[B, T, H m] laid out as `like` is shaped."""
    if like.dim() == 3:
        return y
    return y.unflatten(2, (like.shape[1], like.shape[3])).transpose(1, 2).contiguous()


def _valid(s, T, B):
    t = torch.arange(T, device="cuda")
    n = s["lengths"]
    return None if n is None else (t[None, :] < n[:, None])[..., None]


def _extended(s, W):
    """The carried inputs before the row's own, and the indices of its last W - 1."""
    x = _rows(s["x"]).float()
    B, T, C = x.shape
    carried = torch.zeros(B, W - 1, C, device="cuda") if s["state"] is None else s["state"].float()
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    last = (n[:, None] + torch.arange(W - 1, device="cuda"))[..., None].expand(B, W - 1, C)
    return torch.cat([carried, x], 1), last


def _plain_conv_fwd(s):
    W = s["case"]["W"]
    xe, last = _extended(s, W)
    B, T = xe.shape[0], xe.shape[1] - W + 1
    y = sum(xe[:, j:j + T] * s["weight"][:, j] for j in range(W)) + s["bias"]
    if s["case"]["act"] == "silu":
        y = y * torch.sigmoid(y)
    ok = _valid(s, T, B)
    y = y if ok is None else torch.where(ok, y, 0.0)
    dt = s["x"].dtype
    return _heads(y.to(dt), s["x"]), xe.gather(1, last).to(dt)


def _plain_conv_bwd(s):
    W = s["case"]["W"]
    xe, last = _extended(s, W)
    B, T = xe.shape[0], xe.shape[1] - W + 1
    w = s["weight"]
    dp = _rows(s["dy"]).float()
    if s["case"]["act"] == "silu":
        p = sum(xe[:, j:j + T] * w[:, j] for j in range(W)) + s["bias"]
        sg = torch.sigmoid(p)
        dp = dp * sg * (1 + p * (1 - sg))
    ok = _valid(s, T, B)
    dp = dp if ok is None else torch.where(ok, dp, 0.0)
    pad = torch.nn.functional.pad
    dxe = sum(pad(dp * w[:, j], (0, 0, j, W - 1 - j)) for j in range(W))
    if s["dstate_out"] is not None:
        dxe = dxe.scatter_add(1, last, s["dstate_out"].float())
    dt = s["x"].dtype
    return dict(dx=_heads(dxe[:, W - 1:].to(dt), s["x"]),
                dweight=torch.stack([(dp * xe[:, j:j + T]).sum((0, 1)) for j in range(W)], 1),
                dbias=dp.sum((0, 1)), dstate=dxe[:, :W - 1].to(dt))


def _plain_conv_step(s):
    at = s["slots"].long()
    x, old = s["x"].float(), s["state"][at].float()
    xe = torch.cat([old, x[:, None]], 1)
    y = (xe * s["weight"].t()).sum(1) + s["bias"]
    if s["case"]["act"] == "silu":
        y = y * torch.sigmoid(y)
    s["state"][at] = xe[:, 1:].to(s["x"].dtype)
    return y.to(s["x"].dtype), s["state"]


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, by doubling."""
    T, k = a.shape[1], 1
    while k < T:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        if 2 * k < T:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _spread(v, D):
    """[..., G, N] for every channel of its group: [..., D, N]."""
    return v.float().repeat_interleave(D // v.shape[-2], -2)


def _step_sizes(s):
    """softplus(delta + bias) and its derivative, masked tokens without a step."""
    raw = s["delta"].float() + s["delta_bias"]
    step = raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))
    slope = torch.sigmoid(raw)
    ok = _valid(s, raw.shape[1], raw.shape[0]) if "lengths" in s else None
    return (step, slope) if ok is None else (torch.where(ok, step, 0.0),
                                             torch.where(ok, slope, 0.0))


def _states(s, step):
    """Every decay [B, T, D, N] and every state."""
    D = step.shape[-1]
    a = torch.exp(step[..., None] * s["A"])
    b = (step * s["u"].float())[..., None] * _spread(s["Bm"], D)
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    return a, _recur(a, b)


def _plain_scan_fwd(s):
    step, _ = _step_sizes(s)
    B, T, D = step.shape
    _, h = _states(s, step)
    y = (h * _spread(s["Cm"], D)).sum(-1) + s["D"] * s["u"].float()
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    ok = _valid(s, T, B)
    y = y if ok is None else torch.where(ok, y, 0.0)
    return y.to(s["u"].dtype), h[:, -1].clone()


def _plain_scan_bwd(s):
    step, slope = _step_sizes(s)
    B, T, D = step.shape
    G, N = s["Bm"].shape[-2:]
    dt = s["u"].dtype
    u, A = s["u"].float(), s["A"]
    a, h = _states(s, step)
    C = _spread(s["Cm"], D)
    dy = s["dy"].float()
    ok = _valid(s, T, B)
    dy = dy if ok is None else torch.where(ok, dy, 0.0)
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        y = (h * C).sum(-1) + s["D"] * u
        out["dz"] = (dy * y * sg * (1 + z * (1 - sg))).to(dt)
        dy = dy * z * sg
    out["dC"] = (dy[..., None] * h).view(B, T, G, D // G, N).sum(3).to(dt)
    # adjoints: g_t = C_t dy_t + a_{t+1} g_{t+1}, from the last token back
    g = dy[..., None] * C
    if s["dh_T"] is not None:
        g[:, -1] += s["dh_T"]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _recur(after.flip(1), g.flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None],
                        h[:, :-1]], 1)
    ga = g * a * before
    Bf = _spread(s["Bm"], D)
    gB = (g * Bf).sum(-1)
    dstep = (ga * A).sum(-1) + gB * u
    draw_ = dstep * slope
    out.update(du=(gB * step + s["D"] * dy).to(dt), ddelta=draw_.to(dt),
               dA=(ga * step[..., None]).sum((0, 1)),
               dB=(g * (step * u)[..., None]).view(B, T, G, D // G, N).sum(3).to(dt),
               dD=(dy * u).sum((0, 1)), ddelta_bias=draw_.sum((0, 1)),
               dh0=a[:, 0] * g[:, 0])
    return out


def _plain_scan_step(s):
    at = s["slots"].long()
    step, _ = _step_sizes(s)
    u, D = s["u"].float(), step.shape[-1]
    h = s["h"][at] * torch.exp(step[..., None] * s["A"]) \
        + (step * u)[..., None] * _spread(s["Bm"], D)
    s["h"][at] = h
    y = (h * _spread(s["Cm"], D)).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(s["u"].dtype), s["h"]


def _plain_clip(s):
    total = torch.cat([g.reshape(-1) for g in s["grads"]]).double().square().sum()
    norm = total.sqrt().float()
    scale = (s["max_norm"] / (norm + _CLIP_EPS)).clamp(max=1.0)
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g.float() * scale)
    return norm, s["out"]


# --------------------------------------------------------------------- one pass

def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if not own:
        return {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd,
                "conv_step": _plain_conv_step, "scan_fwd": _plain_scan_fwd,
                "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
                "clip": _plain_clip}[op](s)
    import delta_rule_attention_gb300 as falcon
    if op == "conv_fwd":
        return falcon.falcon_short_conv_fwd(s["x"], s["weight"], bias=s["bias"],
                                            state=s["state"], lengths=s["lengths"],
                                            activation=case["act"])
    if op == "conv_bwd":
        return falcon.falcon_short_conv_bwd(s["x"], s["weight"], s["dy"], bias=s["bias"],
                                            state=s["state"], lengths=s["lengths"],
                                            dstate_out=s["dstate_out"], activation=case["act"])
    if op == "conv_step":
        y = falcon.falcon_short_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"],
                                          slots=s["slots"], activation=case["act"])
        return y, s["state"]
    if op == "scan_fwd":
        return falcon.falcon_selective_scan_fwd(
            s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], D=s["D"], z=s["z"],
            delta_bias=s["delta_bias"], h0=s["h0"], lengths=s["lengths"])
    if op == "scan_bwd":
        g = falcon.falcon_selective_scan_bwd(
            s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["dy"], D=s["D"], z=s["z"],
            delta_bias=s["delta_bias"], h0=s["h0"], lengths=s["lengths"], dh_T=s["dh_T"])
        return {k: v for k, v in g.items() if v is not None}
    if op == "scan_step":
        y = falcon.falcon_selective_scan_step(
            s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["h"], D=s["D"], z=s["z"],
            delta_bias=s["delta_bias"], slots=s["slots"])
        return y, s["h"]
    norm = falcon.falcon_clip_grad_norm(s["grads"], s["max_norm"], out=s["outs"], eps=_CLIP_EPS)
    return norm, s["out"]


# ------------------------------------------------------------------------- work

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("conv_fwd", "conv_bwd"):
        C, W = case["H"] * case["m"], case["W"]
        n = case["B"] * case["T"] * C
        tail = case["B"] * (W - 1) * C * e * (2 if case["state"] else 1)
        if op == "conv_fwd":
            return dict(bytes=2 * n * e + tail + C * (W + 1) * 4, flops=n * (2 * W + 5))
        return dict(bytes=3 * n * e + 2 * tail + 2 * C * (W + 1) * 4, flops=n * (6 * W + 12))
    if op == "conv_step":
        N, C, W = case["N"], case["C"], case["W"]
        return dict(bytes=N * C * e * 2 * W + C * (W + 1) * 4, flops=N * C * (2 * W + 5))
    if op in ("scan_fwd", "scan_bwd"):
        B, T, D, G, N = (case[k] for k in ("B", "T", "D", "G", "N"))
        rows, states = B * T, B * D * N * 4 * (2 if case["state"] else 1)
        gate = 1 if case["gate"] else 0
        if op == "scan_fwd":
            return dict(bytes=rows * (D * (3 + gate) + 2 * G * N) * e + states + D * (N + 2) * 4,
                        flops=rows * D * (8 * N + 12))
        return dict(bytes=rows * (D * (5 + 2 * gate) + 4 * G * N) * e + 2 * states
                    + 2 * D * (N + 2) * 4, flops=rows * D * (24 * N + 30))
    if op == "scan_step":
        N, D, G, S = (case[k] for k in ("N", "D", "G", "S"))
        return dict(bytes=N * (D * (3 + (1 if case["gate"] else 0)) + 2 * G * S) * e
                    + 2 * N * D * S * 4 + D * (S + 2) * 4, flops=N * D * (8 * S + 12))
    n = sum(math.prod(sh) for sh in _clip_shapes(case))
    return dict(bytes=2 * n * e, flops=3 * n)


# ------------------------------------------------- the definitions in 64 bits

def _f64(t):
    return None if t is None else t.double()


def _silu64(v):
    return v / (1 + torch.exp(-v))


def _dsilu64(v):
    q = 1 / (1 + torch.exp(-v))
    return q + v * q * (1 - q)


def _exact_conv(s, want_grads):
    """Row by row: each row's inputs are its carried ones and its own first n."""
    case = s["case"]
    W, H = case["W"], case["H"]
    x = _f64(s["x"])
    x = x if H == 1 else x.permute(0, 2, 1, 3).reshape(x.shape[0], x.shape[2], -1)
    B, T, C = x.shape
    w, bias = _f64(s["weight"]), _f64(s["bias"])
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    y, tail = torch.zeros_like(x), x.new_zeros(B, W - 1, C)
    dx, dst = torch.zeros_like(x), x.new_zeros(B, W - 1, C)
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    if want_grads:
        dy = _f64(s["dy"])
        dy = dy if H == 1 else dy.permute(0, 2, 1, 3).reshape(B, T, C)
    for b in range(B):
        before = x.new_zeros(W - 1, C) if s["state"] is None else _f64(s["state"][b])
        row = torch.cat([before, x[b, :n[b]]])
        tail[b] = row[len(row) - (W - 1):]
        windows = row.unfold(0, W, 1) if n[b] else row.new_zeros(0, C, W)  # [n, C, W]
        pre = torch.einsum("tcj,cj->tc", windows, w) + bias
        y[b, :n[b]] = _silu64(pre) if case["act"] == "silu" else pre
        if want_grads:
            dp = dy[b, :n[b]] * (_dsilu64(pre) if case["act"] == "silu" else 1.0)
            dw += torch.einsum("tc,tcj->cj", dp, windows)
            db += dp.sum(0)
            drow = torch.zeros_like(row)
            for j in range(W):
                drow[j:j + n[b]] += dp * w[:, j]
            if s["dstate_out"] is not None:
                drow[len(row) - (W - 1):] += _f64(s["dstate_out"][b])
            dst[b], dx[b, :n[b]] = drow[:W - 1], drow[W - 1:]
    back = (lambda t: t if H == 1 else t.view(B, T, H, -1).permute(0, 2, 1, 3))
    return dict(dx=back(dx), dweight=dw, dbias=db, dstate=dst) if want_grads else (back(y), tail)


def _exact_scan(s, want_grads):
    case = s["case"]
    B, T, D, G, N = (case[k] for k in ("B", "T", "D", "G", "N"))
    A, Dw, bias = _f64(s["A"]), _f64(s["D"]), _f64(s["delta_bias"])
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    R = D // G
    h = torch.zeros(B, D, N, device="cuda", dtype=torch.float64)
    if s["h0"] is not None:
        h = _f64(s["h0"]).clone()
    y = torch.zeros(B, T, D, device="cuda", dtype=torch.float64)
    kept = []
    for t in range(T):
        on = (t < n).double()[:, None]
        st = torch.log(1 + torch.exp(_f64(s["delta"][:, t]) + bias)) * on
        ut = _f64(s["u"][:, t])
        if want_grads:
            kept.append(h)
        Bt = _f64(s["Bm"][:, t])[:, :, None, :].expand(B, G, R, N).reshape(B, D, N)
        Ct = _f64(s["Cm"][:, t])[:, :, None, :].expand(B, G, R, N).reshape(B, D, N)
        h = torch.exp(st[..., None] * A) * h + (st * ut)[..., None] * Bt
        y[:, t] = (torch.einsum("bdn,bdn->bd", h, Ct) + Dw * ut) * on
    if not want_grads:
        if s["z"] is not None:
            y *= _silu64(_f64(s["z"]))
        return y, h
    g = torch.zeros_like(h) if s["dh_T"] is None else _f64(s["dh_T"]).clone()
    zero = torch.zeros_like
    du, dd, dz = zero(y), zero(y), zero(y)
    dB = torch.zeros(B, T, G, N, device="cuda", dtype=torch.float64)
    dC, dA, dD, dbias = zero(dB), zero(A), zero(Dw), zero(bias)
    for t in reversed(range(T)):
        on = (t < n).double()[:, None]
        raw = _f64(s["delta"][:, t]) + bias
        st, ut, dyt = torch.log(1 + torch.exp(raw)) * on, _f64(s["u"][:, t]), _f64(s["dy"][:, t]) * on
        if s["z"] is not None:
            zt = _f64(s["z"][:, t])
            dz[:, t] = dyt * y[:, t] * _dsilu64(zt)
            dyt = dyt * _silu64(zt)
        Bt = _f64(s["Bm"][:, t])[:, :, None, :].expand(B, G, R, N).reshape(B, D, N)
        Ct = _f64(s["Cm"][:, t])[:, :, None, :].expand(B, G, R, N).reshape(B, D, N)
        old = kept.pop()
        a = torch.exp(st[..., None] * A)
        now = a * old + (st * ut)[..., None] * Bt
        dC[:, t] = (dyt[..., None] * now).view(B, G, R, N).sum(2)
        g = g + dyt[..., None] * Ct
        dB[:, t] = (g * (st * ut)[..., None]).view(B, G, R, N).sum(2)
        du[:, t] = (g * Bt).sum(-1) * st + Dw * dyt
        through = g * a * old
        dst = (through * A).sum(-1) + (g * Bt).sum(-1) * ut
        dd[:, t] = dst * on / (1 + torch.exp(-raw))
        dbias += dd[:, t].sum(0)
        dA += (through * st[..., None]).sum(0)
        dD += (dyt * ut).sum(0)
        g = g * a
    out = dict(du=du, ddelta=dd, dA=dA, dB=dB, dC=dC, dD=dD, ddelta_bias=dbias, dh0=g)
    if s["z"] is not None:
        out["dz"] = dz
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("conv_fwd", "conv_bwd"):
        return _exact_conv(s, op == "conv_bwd")
    if op == "conv_step":
        y, pool = [], s["state"].double()
        for i, at in enumerate(s["slots"].tolist()):
            row = torch.cat([pool[at], s["x"][i:i + 1].double()])
            pre = (row * s["weight"].double().t()).sum(0) + s["bias"].double()
            y.append(_silu64(pre) if case["act"] == "silu" else pre)
            pool[at] = row[1:]
        return torch.stack(y), pool
    if op in ("scan_fwd", "scan_bwd"):
        return _exact_scan(s, op == "scan_bwd")
    if op == "scan_step":
        N, D, G, S = (case[k] for k in ("N", "D", "G", "S"))
        at = s["slots"].long()
        st = torch.log(1 + torch.exp(_f64(s["delta"]) + _f64(s["delta_bias"])))
        wide = lambda v: _f64(v)[:, :, None, :].expand(N, G, D // G, S).reshape(N, D, S)  # noqa: E731
        pool = s["h"].double()
        h = torch.exp(st[..., None] * _f64(s["A"])) * pool[at] \
            + (st * _f64(s["u"]))[..., None] * wide(s["Bm"])
        pool[at] = h
        y = torch.einsum("bdn,bdn->bd", h, wide(s["Cm"])) + _f64(s["D"]) * _f64(s["u"])
        return (y if s["z"] is None else y * _silu64(_f64(s["z"]))), pool
    norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
    scale = min(1.0, s["max_norm"] / (norm + _CLIP_EPS))
    out = s["out"].double()
    where = s["out"].data_ptr()
    for g, o in zip(s["grads"], s["outs"]):
        first = (o.data_ptr() - where) // o.element_size()
        out[first:first + g.numel()] = g.double().reshape(-1) * scale
    return torch.tensor(norm, dtype=torch.float64), out
