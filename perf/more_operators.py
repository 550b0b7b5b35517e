"""The operators of a linear attention block with a fixed decay a head, as cases to time
and to check.

Two operators, each in the forms that a program needs:

  decay attention   S_t = gamma S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, one
                    gamma = exp(log_decay) a head: over prompts, its gradient, and one
                    token of many sequences;
  gated norm        out = x + scale * act(z) * norm(h) w around a block, the norm over
                    each head or over all channels, and the next block's norm(out) w'
                    in the same pass; its gradient.

`own` False computes each in plain torch operations, `own` True through the
package's entry points.  `exact` computes the same from the definitions in
64 bits, token by token.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6


def listed():
    return [
        # A batch of training sequences or prompts of a language-model layer.
        dict(name="decay prompt", op="decay_fwd", dtype="bf16", B=8, H=12, T=2048, m=64, dv=64,
             state=False, ragged=False, rows=True),
        # One long document, few and wide heads.
        dict(name="decay long", op="decay_fwd", dtype="bf16", B=1, H=16, T=65536, m=128, dv=128,
             state=False, ragged=False, rows=True),
        # Continued prompts of uneven lengths, padded, in full precision.
        dict(name="decay ragged f32", op="decay_fwd", dtype="f32", B=5, H=3, T=777, m=64, dv=48,
             state=True, ragged=True, rows=False),
        # The training step's gradient.
        dict(name="decay backward", op="decay_bwd", dtype="bf16", B=8, H=12, T=2048, m=64, dv=64,
             state=False, ragged=False, rows=True),
        # Gradients through carried states, uneven lengths, values wider than keys.
        dict(name="decay backward ragged", op="decay_bwd", dtype="bf16", B=3, H=8, T=1531, m=64,
             dv=128, state=True, ragged=True, rows=False),
        # One token of a large serving batch, states in a pool of slots.
        dict(name="decay step", op="decay_step", dtype="bf16", N=256, H=32, m=128, dv=128),
        # One token of a few sequences: latency.
        dict(name="decay step few", op="decay_step", dtype="bf16", N=2, H=12, m=64, dv=64),
        # Between the attention and its output projection: every head normalised, gated,
        # and turned from head-major tensors into rows.
        dict(name="norm after heads", op="norm_fwd", dtype="bf16", B=8, H=12, T=2048, m=64,
             gate="silu", residual=False, scale=False, next=False, ragged=False, heads=True),
        # Between two blocks: one's output normalised, scaled and added, the next's input.
        dict(name="norm between blocks", op="norm_fwd", dtype="bf16", B=8, H=1, T=2048, m=2048,
             gate="none", residual=True, scale=True, next=True, ragged=False, heads=False),
        # The same for one token of a serving batch: latency.
        dict(name="norm step", op="norm_fwd", dtype="bf16", B=256, H=1, T=1, m=4096,
             gate="none", residual=True, scale=True, next=True, ragged=False, heads=False),
        # The training step's gradient between two blocks.
        dict(name="norm backward", op="norm_bwd", dtype="bf16", B=8, H=1, T=2048, m=2048,
             gate="none", residual=True, scale=True, next=True, ragged=False, heads=False),
        # Every part of it at once, with odd sizes and uneven lengths.
        dict(name="norm backward odd", op="norm_bwd", dtype="f32", B=5, H=3, T=777, m=111,
             gate="sigmoid", residual=True, scale=True, next=True, ragged=True, heads=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decay_fwd", "decay_fwd", "decay_bwd", "decay_bwd", "decay_step",
                     "norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "decay_step":
        H, m, dv = _log_int(rng, 1, 32), rng.choice([16, 32, 64, 64, 128, 40]), \
            rng.choice([16, 32, 64, 64, 128, 37])
        return dict(op=op, dtype=dtype, N=_log_int(rng, 1, min(2048, (1 << 27) // (H * m * dv))),
                    H=H, m=m, dv=dv)
    if op.startswith("decay"):
        m, dv = (rng.choice([16, 32, 64, 64, 64, 128, 128, 48, 80, 37]) for _ in range(2))
        H = rng.choice([1, 2, 4, 8, 12, 16, 5])
        T = _log_int(rng, 1, 32768)
        most = (1 << 24 if dtype == "f32" or op == "decay_bwd" else 1 << 26) // (H * max(m, dv))
        T = min(T, most)
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, max(1, min(32, most // T))), H=H, T=T,
                    m=m, dv=dv, state=rng.random() < 0.5, ragged=rng.random() < 0.4,
                    rows=rng.random() < 0.5)
    H = rng.choice([1, 1, 12, 16, 5])
    m = _log_int(rng, 64, 8192) if H == 1 else rng.choice([16, 32, 64, 128, 111])
    if H == 1 and rng.random() < 0.6:
        m = (m + 7) // 8 * 8
    T = _log_int(rng, 1, 16384)
    most = (1 << 25) // (H * m)
    T = min(T, most)
    gate = rng.choice(["none", "silu", "silu", "sigmoid", "identity"])
    residual = rng.random() < 0.6
    return dict(op=op, dtype=dtype, B=_log_int(rng, 1, max(1, min(256, most // T))), H=H, T=T, m=m,
                gate=gate, residual=residual, scale=residual and rng.random() < 0.5,
                next=residual and rng.random() < 0.7, ragged=rng.random() < 0.3,
                heads=H > 1 and rng.random() < 0.6)


# --------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _lengths(g, case):
    """Uneven lengths, 0 and T among them where there are rows enough."""
    n = torch.randint(0, case["T"] + 1, (case["B"],), generator=g, device="cuda")
    n[0] = case["T"]
    if case["B"] > 2:
        n[1] = 0
    return n.to(torch.int32)


def _log_decays(g, H):
    """Heads from fast to slow, as such layers are set up: a token's weight halves within
    about 1.4 to 2800 tokens."""
    at = torch.rand(H, generator=g, device="cuda") * 0.5 + torch.arange(H, device="cuda")
    return -torch.exp2(-1.0 - 11.0 * at / max(H - 0.5, 1.0))


def _prepare_decay(case, g, dt):
    B, H, T, m, dv = (case[k] for k in ("B", "H", "T", "m", "dv"))
    s = dict(case=case, log_decay=_log_decays(g, H))
    if case["rows"]:  # parts of one projection's rows [B, T, H (2 m + dv)]
        qkv = _randn(g, B, T, H * (2 * m + dv), dtype=dt)
        part = lambda a, w: qkv[..., a:a + H * w].unflatten(2, (H, w)).transpose(1, 2)  # noqa: E731
        s["q"], s["k"], s["v"] = part(0, m), part(H * m, m), part(2 * H * m, dv)
    else:
        s["q"], s["k"], s["v"] = (_randn(g, B, H, T, w, dtype=dt) for w in (m, m, dv))
    s["S0"] = _randn(g, B, H, m, dv) if case["state"] else None
    s["lengths"] = _lengths(g, case) if case["ragged"] else None
    if case["op"] == "decay_bwd":
        s["do"] = _randn(g, B, H, T, dv, dtype=dt)
        s["dS_T"] = _randn(g, B, H, m, dv) if case["state"] else None
    return s


def _prepare_step(case, g, dt):
    N, H, m, dv = (case[k] for k in ("N", "H", "m", "dv"))
    qkv = _randn(g, N, H * (2 * m + dv), dtype=dt)
    part = lambda a, w: qkv[:, a:a + H * w].unflatten(1, (H, w))  # noqa: E731
    pool = N + N // 16 + 1
    return dict(case=case, log_decay=_log_decays(g, H), q=part(0, m), k=part(H * m, m),
                v=part(2 * H * m, dv), S=_randn(g, pool, H, m, dv),
                slots=torch.randperm(pool, generator=g, device="cuda")[:N].to(torch.int32))


def _prepare_norm(case, g, dt):
    B, H, T, m = (case[k] for k in ("B", "H", "T", "m"))
    D = H * m
    s = dict(case=case)
    if case["heads"]:
        s["h"] = _randn(g, B, H, T, m, dtype=dt)  # as an attention writes it
    else:
        h = _randn(g, B, T, D, dtype=dt)
        s["h"] = h if H == 1 else h.unflatten(2, (H, m)).transpose(1, 2)
    # the gate beside other parts of a projection's rows
    s["z"] = _randn(g, B, T, 2 * D, dtype=dt)[..., D:] if case["gate"] != "none" else None
    s["weight"] = 1.0 + 0.1 * _randn(g, D)
    s["scale"] = 0.3 + 0.05 * _randn(g, D) if case["scale"] else None
    s["x"] = 2.0 * _randn(g, B, T, D, dtype=dt) if case["residual"] else None
    s["next_weight"] = 1.0 + 0.1 * _randn(g, D) if case["next"] else None
    s["lengths"] = _lengths(g, case) if case["ragged"] else None
    if case["op"] == "norm_bwd":
        # the stored output of the forward pass; any values will do where it had no residual
        s["out"] = 2.0 * _randn(g, B, T, D, dtype=dt) if case["next"] else None
        s["dout"] = _randn(g, B, T, D, dtype=dt)
        s["dnext"] = _randn(g, B, T, D, dtype=dt) if case["next"] else None
    return s


def prepare(case, seed):
    g = _gen(seed)
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "decay_step":
        return _prepare_step(case, g, dt)
    return (_prepare_decay if case["op"].startswith("decay") else _prepare_norm)(case, g, dt)


# ---------------------------------------------------------------- plain forms

def _on(s, T):
    """Which tokens [B, T] a padded batch holds; None: all."""
    n = s["lengths"]
    return None if n is None else torch.arange(T, device="cuda")[None, :] < n[:, None]


def _kept(t, on):
    """[B, H, T, *] in 32 bits, zero where there is no token."""
    t = t.float()
    return t if on is None else torch.where(on[:, None, :, None], t, 0.0)


def _counts(s, B, T):
    return torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()


def _powers(g, n):
    """gamma^n for every head: [H, *n.shape]."""
    return torch.exp(g.view(-1, *[1] * n.dim()) * n)


def _read(q, k, v, g):
    """sum_{j <= t} gamma^(t - j) (q_t . k_j) v_j, chunk by chunk and between chunks."""
    B, H, T, _ = q.shape
    C = max(64, 1 << (max(T - 1, 1).bit_length() + 1) // 2)
    n = (T + C - 1) // C
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, n * C - T)).unflatten(2, (n, C))
               for t in (q, k, v))
    i = torch.arange(C, device="cuda")
    gap = i[:, None] - i
    within = torch.where(gap >= 0, _powers(g, gap.clamp(min=0)), 0.0)
    o = (q @ k.transpose(-1, -2) * within[:, None]) @ v
    if n > 1:
        grown = (k * _powers(g, C - 1 - i)[:, None, :, None]).transpose(-1, -2) @ v
        c = torch.arange(n, device="cuda")
        gap = c[:, None] - 1 - c
        between = torch.where(gap >= 0, _powers(g, C * gap.clamp(min=0)), 0.0)
        entering = (between @ grown.flatten(3)).view_as(grown)
        o = o + (q * _powers(g, i + 1)[:, None, :, None]) @ entering
    return o.flatten(2, 3)[:, :, :T]


def _plain_decay_fwd(s):
    B, H, T, m = s["q"].shape
    on, g = _on(s, T), s["log_decay"]
    q, k, v = (_kept(s[x], on) for x in "qkv")
    t, n = torch.arange(T, device="cuda"), _counts(s, B, T)
    o = _read(q, k, v, g)
    left = (n[:, None] - 1 - t).clamp(min=0)
    S = (k * _powers(g, left).transpose(0, 1)[..., None]).transpose(-1, -2) @ v
    if s["S0"] is not None:
        o = o + (q * _powers(g, t + 1)[None, :, :, None]) @ s["S0"]
        S = S + _powers(g, n).t()[..., None, None] * s["S0"]
    return (o * m ** -0.5).to(s["q"].dtype), S


def _plain_decay_bwd(s):
    B, H, T, m = s["q"].shape
    on, g, dt = _on(s, T), s["log_decay"], s["q"].dtype
    q, k, v, do = (_kept(s[x], on) for x in ("q", "k", "v", "do"))
    do = do * m ** -0.5
    t, n = torch.arange(T, device="cuda"), _counts(s, B, T)
    back = lambda a, b, c: _read(a.flip(2), b.flip(2), c.flip(2), g).flip(2)  # noqa: E731
    dq, dk, dv = _read(do, v, k, g), back(v, do, q), back(k, q, do)
    grown = _powers(g, t + 1)[None, :, :, None]
    dS0 = (q * grown).transpose(-1, -2) @ do
    if s["S0"] is not None:
        dq = dq + grown * (do @ s["S0"].transpose(-1, -2))
    if s["dS_T"] is not None:
        left = _powers(g, (n[:, None] - 1 - t).clamp(min=0)).transpose(0, 1)[..., None]
        dk = dk + left * (v @ s["dS_T"].transpose(-1, -2))
        dv = dv + left * (k @ s["dS_T"])
        dS0 = dS0 + _powers(g, n).t()[..., None, None] * s["dS_T"]
    return dict(dq=dq.to(dt), dk=dk.to(dt), dv=dv.to(dt), dS0=dS0)


def _plain_decay_step(s):
    at = s["slots"].long()
    q, k, v = (s[x].float() for x in "qkv")
    S = s["S"][at] * torch.exp(s["log_decay"])[:, None, None] + k[..., None] * v[..., None, :]
    s["S"][at] = S
    o = (S * q[..., None]).sum(-2) * q.shape[-1] ** -0.5
    return o.to(s["q"].dtype), s["S"]


def _act(z, gate):
    return z * torch.sigmoid(z) if gate == "silu" else \
        torch.sigmoid(z) if gate == "sigmoid" else z


def _act_slope(z, gate):
    if gate == "identity":
        return torch.ones_like(z)
    q = torch.sigmoid(z)
    return q * (1 + z * (1 - q)) if gate == "silu" else q * (1 - q)


def _by_head(h):
    """[B, T, D] or [B, H, T, m] in 32 bits as [B, T, H, m]."""
    return h.float().unsqueeze(2) if h.dim() == 3 else h.float().transpose(1, 2)


def _scaled_to_one(h):
    return torch.rsqrt(h.square().mean(-1, keepdim=True) + _EPS)


def _held(t, on):
    return t if on is None else torch.where(on[..., None], t, 0.0)


def _plain_norm_fwd(s):
    case, dt = s["case"], s["h"].dtype
    h = _by_head(s["h"])
    on = _on(s, h.shape[1])
    y = (h * _scaled_to_one(h)).flatten(2) * s["weight"]
    if s["z"] is not None:
        y = y * _act(s["z"].float(), case["gate"])
    if s["scale"] is not None:
        y = y * s["scale"]
    if s["x"] is not None:
        y = y + s["x"].float()
    y = _held(y, on)
    if s["next_weight"] is None:
        return y.to(dt)
    return y.to(dt), (y * _scaled_to_one(y) * s["next_weight"]).to(dt)


def _norm_back(d, h, r):
    """Through h r, r = rsqrt(mean h^2 + eps): r (d - h r mean(d h r))."""
    return r * (d - h * r * (d * h * r).mean(-1, keepdim=True))


def _plain_norm_bwd(s):
    case, dt = s["case"], s["h"].dtype
    h = _by_head(s["h"])
    B, T, H, m = h.shape
    on = _on(s, T)
    out = {}
    d = _held(s["dout"].float(), on)
    if s["next_weight"] is not None:
        dn, y = _held(s["dnext"].float(), on), _held(s["out"].float(), on)
        r = _scaled_to_one(y)
        out["dnext_weight"] = (dn * y * r).sum((0, 1))
        d = d + _norm_back(dn * s["next_weight"], y, r)
    if s["x"] is not None:
        out["dx"] = d.to(dt)
    h = h if on is None else torch.where(on[..., None, None], h, 0.0)
    r = _scaled_to_one(h)
    normed = (h * r).flatten(2)
    g = s["weight"]
    if s["scale"] is not None:
        g = g * s["scale"]
    gate = 1.0
    if s["z"] is not None:
        z = _held(s["z"].float(), on)
        gate = _act(z, case["gate"])
        out["dz"] = (d * g * normed * _act_slope(z, case["gate"])).to(dt)
    each = (d * gate * normed).sum((0, 1))
    out["dweight"] = each if s["scale"] is None else each * s["scale"]
    if s["scale"] is not None:
        out["dscale"] = each * s["weight"]
    dh = _norm_back((d * gate * g).unflatten(2, (H, m)), h, r)
    out["dh"] = (dh[:, :, 0] if s["h"].dim() == 3 else dh.transpose(1, 2).contiguous()).to(dt)
    return out


# --------------------------------------------------------------------- one pass

def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if not own:
        return {"decay_fwd": _plain_decay_fwd, "decay_bwd": _plain_decay_bwd,
                "decay_step": _plain_decay_step, "norm_fwd": _plain_norm_fwd,
                "norm_bwd": _plain_norm_bwd}[op](s)
    import delta_rule_attention_gb300 as falcon
    if op == "decay_fwd":
        return falcon.falcon_decay_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], S0=s["S0"],
                                            lengths=s["lengths"])
    if op == "decay_bwd":
        return falcon.falcon_decay_attn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"],
                                            S0=s["S0"], lengths=s["lengths"], dS_T=s["dS_T"])
    if op == "decay_step":
        o = falcon.falcon_decay_attn_step(s["q"], s["k"], s["v"], s["log_decay"], s["S"],
                                          slots=s["slots"])
        return o, s["S"]
    gate = "silu" if case["gate"] == "none" else case["gate"]
    if op == "norm_fwd":
        y, u = falcon.falcon_gated_norm_fwd(
            s["h"], weight=s["weight"], z=s["z"], gate=gate, scale=s["scale"], x=s["x"],
            next_weight=s["next_weight"], lengths=s["lengths"], eps=_EPS)
        return y if u is None else (y, u)
    g = falcon.falcon_gated_norm_bwd(
        s["h"], s["dout"], dnext=s["dnext"], out=s["out"], weight=s["weight"], z=s["z"], gate=gate,
        scale=s["scale"], residual=case["residual"], next_weight=s["next_weight"],
        lengths=s["lengths"], eps=_EPS)
    return {k: v for k, v in g.items() if v is not None}


# ------------------------------------------------------------------------- work

def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "decay_step":
        N, H, m, dv = (case[k] for k in ("N", "H", "m", "dv"))
        return dict(bytes=N * H * (e * 2 * (m + dv) + 8 * m * dv), flops=5 * N * H * m * dv)
    if op.startswith("decay"):
        B, H, T, m, dv = (case[k] for k in ("B", "H", "T", "m", "dv"))
        state = 4 * B * H * m * dv
        if op == "decay_fwd":
            return dict(bytes=e * B * H * T * 2 * (m + dv) + state * (2 if case["state"] else 1),
                        flops=B * H * T * 4 * m * dv)
        return dict(bytes=e * B * H * T * (4 * m + 3 * dv) + state * (3 if case["state"] else 1),
                    flops=B * H * T * 10 * m * dv)
    D = case["H"] * case["m"]
    n = case["B"] * case["T"] * D
    z, x, u = case["gate"] != "none", case["residual"], case["next"]
    params = 4 * D * (1 + case["scale"] + u)
    if op == "norm_fwd":
        return dict(bytes=e * n * (2 + z + x + u) + params, flops=n * (6 + 6 * z + 2 * x + 4 * u))
    return dict(bytes=e * n * (3 + 2 * z + x + 2 * u) + 2 * params,
                flops=n * (14 + 12 * z + 12 * u))


# ------------------------------------------------- the definitions in 64 bits

def _exact_decay(s, want_grads):
    """Token by token: the state forward, and its adjoint back."""
    B, H, T, m = s["q"].shape
    dv = s["v"].shape[-1]
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    n = torch.tensor(n, device="cuda")
    gamma = s["log_decay"].double().exp().view(1, H, 1, 1)
    q, k, v = (s[x].double() for x in "qkv")
    scale = 1 / math.sqrt(m)
    S = torch.zeros(B, H, m, dv, device="cuda", dtype=torch.float64)
    if s["S0"] is not None:
        S += s["S0"]
    o = torch.zeros_like(v)
    dq = torch.zeros_like(q)
    for t in range(T):
        on = (t < n).view(B, 1, 1, 1)
        S = torch.where(on, gamma * S + k[:, :, t, :, None] * v[:, :, t, None, :], S)
        if want_grads:
            dq[:, :, t] = torch.einsum("bhmd,bhd->bhm", S, s["do"][:, :, t].double()) * on[..., 0]
        else:
            o[:, :, t] = torch.einsum("bhmd,bhm->bhd", S, q[:, :, t]) * on[..., 0]
    if not want_grads:
        return o * scale, S
    G = torch.zeros_like(S)
    if s["dS_T"] is not None:
        G += s["dS_T"]
    dk, dv_ = torch.zeros_like(k), torch.zeros_like(v)
    for t in reversed(range(T)):
        on = (t < n).view(B, 1, 1, 1)
        more = G + scale * q[:, :, t, :, None] * s["do"][:, :, t, None, :].double()
        dk[:, :, t] = torch.einsum("bhmd,bhd->bhm", more, v[:, :, t]) * on[..., 0]
        dv_[:, :, t] = torch.einsum("bhmd,bhm->bhd", more, k[:, :, t]) * on[..., 0]
        G = torch.where(on, gamma * more, G)
    return dict(dq=dq * scale, dk=dk, dv=dv_, dS0=G)


def _gate64(z, gate):
    p = 1 / (1 + torch.exp(-z))
    return dict(silu=(z * p, p + z * p * (1 - p)), sigmoid=(p, p * (1 - p)),
                identity=(z, torch.ones_like(z)))[gate]


def _exact_norm(s, want_grads):
    """Over the tokens that the batch holds, as one list of rows."""
    case = s["case"]
    B, H, T, m = (case[k] for k in ("B", "H", "T", "m"))
    D = H * m
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    at = torch.tensor([b * T + t for b in range(B) for t in range(n[b])], device="cuda",
                      dtype=torch.long)
    rows = lambda t: t.reshape(B * T, D)[at].double()  # noqa: E731

    def whole(r):
        full = torch.zeros(B * T, D, device="cuda", dtype=torch.float64)
        full[at] = r
        return full.view(B, T, D)

    h = rows(s["h"] if H == 1 and s["h"].dim() == 3 else s["h"].permute(0, 2, 1, 3))
    size = torch.sqrt((h.view(-1, H, m) ** 2).sum(-1) / m + _EPS)[..., None]
    normed = (h.view(-1, H, m) / size).view(-1, D)
    w = s["weight"].double()
    a = s["scale"].double() if s["scale"] is not None else torch.ones_like(w)
    g, slope = (_gate64(rows(s["z"]), case["gate"]) if s["z"] is not None
                else (torch.ones_like(h), None))
    if not want_grads:
        y = normed * w * g * a
        if s["x"] is not None:
            y = y + rows(s["x"])
        if s["next_weight"] is None:
            return whole(y)
        u = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / D + _EPS) * s["next_weight"].double()
        return whole(y), whole(u)
    d = rows(s["dout"])
    out = {}
    if s["next_weight"] is not None:
        y, dn = rows(s["out"]), rows(s["dnext"])
        big = torch.sqrt((y ** 2).sum(-1, keepdim=True) / D + _EPS)
        out["dnext_weight"] = (dn * y / big).sum(0)
        e = dn * s["next_weight"].double()
        d = d + e / big - y * (e * y).sum(-1, keepdim=True) / (D * big ** 3)
    if s["x"] is not None:
        out["dx"] = whole(d)
    if s["z"] is not None:
        out["dz"] = whole(d * a * w * normed * slope)
    out["dweight"] = (d * a * g * normed).sum(0)
    if s["scale"] is not None:
        out["dscale"] = (d * g * w * normed).sum(0)
    f, h = (d * a * g * w).view(-1, H, m), h.view(-1, H, m)
    dh = f / size - h * (f * h).sum(-1, keepdim=True) / (m * size ** 3)
    dh = whole(dh.reshape(-1, D))
    out["dh"] = dh if s["h"].dim() == 3 else dh.view(B, T, H, m).permute(0, 2, 1, 3)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("decay_fwd", "decay_bwd"):
        return _exact_decay(s, op == "decay_bwd")
    if op == "decay_step":
        pool, o = s["S"].double(), []
        gamma = s["log_decay"].double().exp()[:, None, None]
        for i, at in enumerate(s["slots"].tolist()):
            pool[at] = gamma * pool[at] + torch.einsum("hm,hd->hmd", s["k"][i].double(),
                                                       s["v"][i].double())
            o.append(torch.einsum("hmd,hm->hd", pool[at], s["q"][i].double()))
        return torch.stack(o) / math.sqrt(case["m"]), pool
    return _exact_norm(s, op == "norm_bwd")
