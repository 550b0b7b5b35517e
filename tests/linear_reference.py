"""Plain 64-bit forms of the linear attention block's operators, token by token, each with
the size of what it sums (every product by its absolute value), from which the tests'
tolerances follow."""
import torch

F64 = torch.float64


def _wide(*ts):
    return [None if t is None else t.detach().cpu().to(F64) for t in ts]


def lengths_of(lengths, B, T):
    if lengths is None:
        return [T] * B
    return [min(max(int(n), 0), T) for n in lengths]


def gammas(log_decay):
    g = log_decay.detach().cpu().to(F64).clamp(max=0)
    return torch.exp(g)


def decay_forward(q, k, v, log_decay, S0=None, lengths=None, scale=None):
    """(o, S_T) of S_t = gamma S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t."""
    q, k, v, S0 = _wide(q, k, v, S0)
    B, H, T, m = q.shape
    scale = m ** -0.5 if scale is None else scale
    n = lengths_of(lengths, B, T)
    gam = gammas(log_decay)[:, None, None]
    o = torch.zeros_like(v)
    S = torch.zeros(B, H, m, v.shape[-1], dtype=F64) if S0 is None else S0.clone()
    for b in range(B):
        for t in range(n[b]):
            S[b] = gam * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * torch.einsum("hmd,hm->hd", S[b], q[b, :, t])
    return o, S


def decay_gradient(q, k, v, log_decay, dO, S0=None, lengths=None, dS_T=None, scale=None):
    """dict of dq, dk, dv, dS0 from the adjoint G_t = scale q_t dO_t^T + gamma G_{t+1}."""
    q, k, v, dO, S0, dS_T = _wide(q, k, v, dO, S0, dS_T)
    B, H, T, m = q.shape
    scale = m ** -0.5 if scale is None else scale
    n = lengths_of(lengths, B, T)
    gam = gammas(log_decay)[:, None, None]
    zero = torch.zeros(B, H, m, v.shape[-1], dtype=F64)
    S = zero.clone() if S0 is None else S0.clone()
    G = zero.clone() if dS_T is None else dS_T.clone()
    dq, dk, dv = (torch.zeros_like(t) for t in (q, k, v))
    for b in range(B):
        for t in range(n[b]):
            S[b] = gam * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            dq[b, :, t] = scale * torch.einsum("hmd,hd->hm", S[b], dO[b, :, t])
        for t in reversed(range(n[b])):
            G[b] = G[b] + scale * q[b, :, t, :, None] * dO[b, :, t, None, :]
            dk[b, :, t] = torch.einsum("hmd,hd->hm", G[b], v[b, :, t])
            dv[b, :, t] = torch.einsum("hmd,hm->hd", G[b], k[b, :, t])
            G[b] = gam * G[b]
    return dict(dq=dq, dk=dk, dv=dv, dS0=G)


def _abs(*ts):
    return [None if t is None else t.detach().abs() for t in ts]


def decay_forward_size(q, k, v, log_decay, S0=None, lengths=None, scale=None):
    q, k, v, S0 = _abs(q, k, v, S0)
    return decay_forward(q, k, v, log_decay, S0, lengths,
                         None if scale is None else abs(scale))


def decay_gradient_size(q, k, v, log_decay, dO, S0=None, lengths=None, dS_T=None, scale=None):
    q, k, v, dO, S0, dS_T = _abs(q, k, v, dO, S0, dS_T)
    return decay_gradient(q, k, v, log_decay, dO, S0, lengths, dS_T,
                          None if scale is None else abs(scale))


def _gate(z, gate):
    if z is None:
        return 1.0, 0.0
    p = torch.sigmoid(z)
    return dict(silu=(z * p, p * (1 + z * (1 - p))), sigmoid=(p, p * (1 - p)),
                identity=(z, torch.ones_like(z)))[gate]


def _rows(h):
    """[B,T,m] or [B,H,T,m] as [B,T,H,m]."""
    return h.unsqueeze(2) if h.dim() == 3 else h.transpose(1, 2)


def _held(t, n):
    """Zeros behind each row's length, whatever stood there."""
    if t is None:
        return None
    on = torch.arange(t.shape[1])[None, :] < torch.tensor(n)[:, None]
    return torch.where(on.view(*on.shape, *[1] * (t.dim() - 2)), t, torch.zeros((), dtype=F64))


def norm_forward(h, weight=None, z=None, gate="silu", scale=None, x=None, next_weight=None,
                 lengths=None, eps=1e-6):
    """((out, next), (their sizes)); next None without next_weight."""
    h, weight, z, scale, x, next_weight = _wide(h, weight, z, scale, x, next_weight)
    B, T = (x.shape[:2] if h is None else _rows(h).shape[:2])
    n = lengths_of(lengths, B, T)
    z, x = _held(z, n), _held(x, n)
    y = size = 0.0
    if h is not None:
        hr = _held(_rows(h), n)
        y = (hr / torch.sqrt(hr.square().mean(-1, keepdim=True) + eps)).flatten(2)
        for f in (weight, scale, _gate(z, gate)[0]):
            if f is not None:
                y = y * f
        size = y.abs() if torch.is_tensor(y) else y
    if x is not None:
        y, size = y + x, size + x.abs()
    y, size = _held(y, n), _held(size, n)
    if next_weight is None:
        return (y, None), (size, None)
    s = torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * next_weight
    # a part of size d in y moves its own quotient, and through the mean all of the row's
    spread = (size * y.abs()).mean(-1, keepdim=True) / (y.square().mean(-1, keepdim=True) + eps)
    return (y, y * s), (size, (size + y.abs() * spread) * s.abs())


def norm_gradient(h, dout, dnext=None, out=None, weight=None, z=None, gate="silu", scale=None,
                  residual=True, next_weight=None, lengths=None, eps=1e-6):
    """(gradients, their sizes) as dicts, by the formulas of the fused pass."""
    h, dout, dnext, out, weight, z, scale, next_weight = _wide(h, dout, dnext, out, weight, z,
                                                               scale, next_weight)
    like = out if h is None else _rows(h)
    n = lengths_of(lengths, *like.shape[:2])
    dout, dnext, out, z = (_held(t, n) for t in (dout, dnext, out, z))
    g, a = {}, {}
    d = torch.zeros_like(dnext) if dout is None else dout
    size = d.abs()
    if next_weight is not None:
        s = torch.rsqrt(out.square().mean(-1, keepdim=True) + eps)
        e = dnext * next_weight
        g["dnext_weight"] = (dnext * out * s).sum((0, 1))
        a["dnext_weight"] = (dnext * out * s).abs().sum((0, 1))
        d = d + s * (e - out * s * s * (e * out).mean(-1, keepdim=True))
        size = size + s * (e.abs() + out.abs() * s * s * (e * out).abs().mean(-1, keepdim=True))
    if residual or h is None:
        g["dx"], a["dx"] = d, size
    if h is None:
        return g, a
    hr = _held(_rows(h), n)
    H = hr.shape[2]
    r = torch.rsqrt(hr.square().mean(-1, keepdim=True) + eps)
    normed = (hr * r).flatten(2)
    act, slope = _gate(z, gate)
    w = 1.0 if weight is None else weight
    c = 1.0 if scale is None else scale
    if z is not None:
        g["dz"] = d * c * w * normed * slope
        # the slope of silu is a sum of two parts
        parts = slope.abs() + (torch.sigmoid(z) * (1 + z.abs()) if gate == "silu" else 0.0)
        a["dz"] = size * abs(c) * abs(w) * normed.abs() * parts
    if weight is not None:
        g["dweight"] = (d * c * act * normed).sum((0, 1))
        a["dweight"] = (size * abs(c) * abs(act) * normed.abs()).sum((0, 1))
    if scale is not None:
        g["dscale"] = (d * w * act * normed).sum((0, 1))
        a["dscale"] = (size * abs(w) * abs(act) * normed.abs()).sum((0, 1))
    f = (d * act * w * c).unflatten(2, (H, -1)) if torch.is_tensor(d * act * w * c) else d
    fa = (size * abs(act) * abs(w) * abs(c)).unflatten(2, (H, -1))
    dh = r * (f - hr * r * r * (f * hr).mean(-1, keepdim=True))
    da = r * (fa + hr.abs() * r * r * (fa * hr.abs()).mean(-1, keepdim=True))
    back = (lambda t: t[:, :, 0]) if h.dim() == 3 else (lambda t: t.transpose(1, 2))
    g["dh"], a["dh"] = back(dh), back(da)
    return g, a
