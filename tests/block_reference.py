"""The selective state space block's operators from their formulas, token by
token in float64 on the CPU: the reference of the block's tests.  Gradients come
from autograd through these loops (checked against differences in
test_block_reference.py)."""
import torch


def f64(t):
    return None if t is None else t.detach().cpu().double()


def silu(v):
    return v * torch.sigmoid(v)


def conv(x, weight, bias=None, state=None, lengths=None, activation="silu"):
    """x [B,T,C] -> (y, state_out)."""
    B, T, C = x.shape
    W = weight.shape[1]
    ys, tails = [], []
    for b in range(B):
        n = T if lengths is None else max(0, min(T, int(lengths[b])))
        before = x.new_zeros(W - 1, C) if state is None else state[b]
        row = torch.cat([before, x[b, :n]])
        out = []
        for t in range(n):
            p = (row[t:t + W] * weight.t()).sum(0)
            if bias is not None:
                p = p + bias
            out.append(silu(p) if activation == "silu" else p)
        out += [x.new_zeros(C)] * (T - n)
        ys.append(torch.stack(out) if out else x.new_zeros(0, C))
        tails.append(row[row.shape[0] - (W - 1):])
    return torch.stack(ys), torch.stack(tails)


def scan(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, h0=None, lengths=None,
         softplus=True):
    """u [B,T,C], Bm, Cm [B,T,G,N] -> (y, h_T)."""
    B, T, C = u.shape
    G, N = Bm.shape[2:]
    ys, hs = [], []
    for b in range(B):
        n = T if lengths is None else max(0, min(T, int(lengths[b])))
        h = u.new_zeros(C, N) if h0 is None else h0[b]
        out = []
        for t in range(n):
            s = delta[b, t] if delta_bias is None else delta[b, t] + delta_bias
            if softplus:
                s = s.clamp(min=0) + torch.log1p(torch.exp(-s.abs()))
            Bt = Bm[b, t].repeat_interleave(C // G, 0)
            Ct = Cm[b, t].repeat_interleave(C // G, 0)
            h = torch.exp(s[:, None] * A) * h + (s * u[b, t])[:, None] * Bt
            o = (Ct * h).sum(1)
            if D is not None:
                o = o + D * u[b, t]
            out.append(o if z is None else o * silu(z[b, t]))
        out += [u.new_zeros(C)] * (T - n)
        ys.append(torch.stack(out) if out else u.new_zeros(0, C))
        hs.append(h)
    return torch.stack(ys), torch.stack(hs)


def gradients(fn, inputs, cotangents):
    """Gradients of sum_i <cotangents_i, fn(**inputs)_i> for every float input."""
    leaves = {k: v.clone().requires_grad_() for k, v in inputs.items()
              if isinstance(v, torch.Tensor) and v.is_floating_point()}
    outs = fn(**{**inputs, **leaves})
    total = sum((o * c).sum() for o, c in zip(outs, cotangents) if c is not None)
    got = torch.autograd.grad(total, list(leaves.values()), allow_unused=True)
    return {k: torch.zeros_like(v) if g is None else g
            for (k, v), g in zip(leaves.items(), got)}


def rel(got, want):
    """||got - want|| / ||want||, and 0 where both vanish."""
    got, want = f64(got).flatten(), f64(want).flatten()
    off, size = float((got - want).norm()), float(want.norm())
    return off / size if size else (0.0 if off == 0.0 else float("inf"))
