"""The block's operators and gradients in float64 with all rows at once, for the
sizes where the token-by-token reference of block_reference.py takes too long.
Checked against it in test_block_vectorised.py."""
import torch


def _mask(lengths, B, T, device):
    if lengths is None:
        return torch.ones(B, T, 1, dtype=torch.float64, device=device)
    t = torch.arange(T, device=device)
    return (t[None, :] < lengths.to(device)[:, None]).double()[..., None]


def _last(lengths, B, T, k, device):
    n = torch.full((B,), T, device=device) if lengths is None else lengths.to(device).long()
    return n.clamp(0, T)[:, None] + torch.arange(k, device=device)


def conv_gradients(x, weight, dy, bias=None, state=None, lengths=None, dstate_out=None,
                   silu=True):
    """dict of dx, dweight, dbias, dstate; float64 inputs, x and dy [B,T,C]."""
    B, T, C = x.shape
    W = weight.shape[1]
    before = x.new_zeros(B, W - 1, C) if state is None else state
    on = _mask(lengths, B, T, x.device)
    xe = torch.cat([before, torch.where(on > 0, x, 0.0)], 1)
    dp = torch.where(on > 0, dy, 0.0)
    if silu:
        p = sum(xe[:, j:j + T] * weight[:, j] for j in range(W))
        p = p if bias is None else p + bias
        s = torch.sigmoid(p)
        dp = dp * (s + p * s * (1 - s))
    dxe = torch.zeros_like(xe)
    for j in range(W):
        dxe[:, j:j + T] += dp * weight[:, j]
    if dstate_out is not None:
        at = _last(lengths, B, T, W - 1, x.device)[..., None].expand(B, W - 1, C)
        dxe.scatter_add_(1, at, dstate_out)
    return dict(dx=dxe[:, W - 1:], dstate=dxe[:, :W - 1], dbias=dp.sum((0, 1)),
                dweight=torch.stack([(dp * xe[:, j:j + T]).sum((0, 1)) for j in range(W)], 1))


def scan_gradients(u, delta, A, Bm, Cm, dy, D=None, z=None, delta_bias=None, h0=None,
                   lengths=None, dh_T=None):
    """dict of du, ddelta, dz, dB, dC, dA, dD, ddelta_bias, dh0; float64 inputs."""
    B, T, C = u.shape
    G, N = Bm.shape[2:]
    on = _mask(lengths, B, T, u.device)
    u, delta, dy = (torch.where(on > 0, t, 0.0) for t in (u, delta, dy))
    Bm, Cm = (torch.where(on[..., None] > 0, t, 0.0) for t in (Bm, Cm))
    raw = delta if delta_bias is None else delta + delta_bias
    step = (raw.clamp(min=0) + torch.log1p(torch.exp(-raw.abs()))) * on
    slope = torch.sigmoid(raw) * on
    skip = A.new_zeros(C) if D is None else D
    wide = lambda v: v.repeat_interleave(C // G, 1)  # noqa: E731
    h = u.new_zeros(B, C, N) if h0 is None else h0
    before, y = [], torch.empty_like(u)
    for t in range(T):
        before.append(h)
        h = torch.exp(step[:, t, :, None] * A) * h \
            + (step[:, t] * u[:, t])[..., None] * wide(Bm[:, t])
        y[:, t] = (wide(Cm[:, t]) * h).sum(-1) + skip * u[:, t]
    out = {}
    if z is not None:
        z = torch.where(on > 0, z, 0.0)
        s = torch.sigmoid(z)
        out["dz"] = dy * y * (s + z * s * (1 - s))
        dy = dy * z * s
    g = torch.zeros_like(h) if dh_T is None else dh_T
    du, dd, dB, dC = (torch.zeros_like(t) for t in (u, u, Bm, Bm))
    dA = torch.zeros_like(A)
    for t in reversed(range(T)):
        a = torch.exp(step[:, t, :, None] * A)
        Bt, Ct, su = wide(Bm[:, t]), wide(Cm[:, t]), step[:, t] * u[:, t]
        now = a * before[t] + su[..., None] * Bt
        dC[:, t] = (dy[:, t, :, None] * now).view(B, G, C // G, N).sum(2)
        g = g + dy[:, t, :, None] * Ct
        dB[:, t] = (g * su[..., None]).view(B, G, C // G, N).sum(2)
        gB = (g * Bt).sum(-1)
        du[:, t] = gB * step[:, t] + skip * dy[:, t]
        w = g * a * before[t]
        dd[:, t] = ((w * A).sum(-1) + gB * u[:, t]) * slope[:, t]
        dA += (w * step[:, t, :, None]).sum(0)
        g = g * a
    out.update(du=du, ddelta=dd, dA=dA, dB=dB, dC=dC, dD=(dy * u).sum((0, 1)),
               ddelta_bias=dd.sum((0, 1)), dh0=g)
    return out
