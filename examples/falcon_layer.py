"""A fast-weight attention layer with the short convolution before q, k and v: a prompt,
the tokens after it, and training steps with the gradients clipped.

    python examples/falcon_layer.py [--width 512] [--heads 8] [--batch 4] [--tokens 1024]

The layer is  q, k, v = heads(conv(W_in r)),  beta = sigmoid(W_b r),  lambda =
softplus(W_l r),  o = Falcon-1A(q, k, v, beta, lambda),  out = W_out o.  The
convolution reads each of q, k and v from the projection's rows and writes it head by
head, as the attention takes it; its gradients go back into one tensor of rows.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import delta_rule_attention_gb300 as falcon  # noqa: E402


class FalconLayer:
    """Parameters of one layer with `heads` heads of `dim` keys and values each."""

    def __init__(self, width, heads, dim=64, taps=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def mat(out, inn, dt=dtype):
            return (torch.randn(out, inn, generator=g, device=device) * inn ** -0.5).to(dt)

        self.heads, self.dim, self.taps, self.dtype = heads, dim, taps, dtype
        channels = heads * dim
        self.w_in, self.w_out = mat(3 * channels, width), mat(width, channels)
        self.w_beta, self.w_lam = (mat(heads, width, torch.float32) for _ in range(2))
        # one filter a channel, for q, k and v
        self.conv_w = torch.randn(3, channels, taps, generator=g, device=device) * taps ** -0.5
        self.conv_b = torch.zeros(3, channels, device=device)

    def _heads(self, rows, i):
        """q, k or v (i = 0, 1, 2) of the projection's rows as [B,H,T,dim]: a view."""
        B, T = rows.shape[:2]
        return rows.view(B, T, 3, self.heads, self.dim)[:, :, i].transpose(1, 2)

    def _gains(self, r):
        beta = torch.sigmoid(r.float() @ self.w_beta.T)
        lam = torch.nn.functional.softplus(r.float() @ self.w_lam.T)
        return beta, lam  # [..., H]

    def prompt(self, r, conv_states=(None, None, None), S=None, x_prev=None):
        """r [B,T,width] -> (out, (conv_states, S, x_last), kept for backward)."""
        rows = r @ self.w_in.T
        qkv, tails = [], []
        for i in range(3):
            y, tail = falcon.falcon_short_conv_fwd(self._heads(rows, i), self.conv_w[i],
                                                   bias=self.conv_b[i], state=conv_states[i])
            qkv.append(y)
            tails.append(tail)
        beta, lam = (t.transpose(1, 2).contiguous() for t in self._gains(r))
        o, S, x_last = falcon.falcon1a_fwd_chunked(*qkv, beta, lam, S0=S, x_prev=x_prev)
        o = o.transpose(1, 2).flatten(2)
        return o @ self.w_out.T, (tails, S, x_last), (r, rows, qkv, beta, lam, o)

    def token(self, r, conv_states, S, x_prev):
        """r [N,width], one token of N sequences; their states are updated in place."""
        N, H = r.shape[0], self.heads
        rows = (r @ self.w_in.T).view(N, 3, H * self.dim)
        q, k, v = (falcon.falcon_short_conv_step(rows[:, i], self.conv_w[i], conv_states[i],
                                                 bias=self.conv_b[i]).view(N * H, self.dim)
                   for i in range(3))
        beta, lam = (t.reshape(N * H) for t in self._gains(r))
        o = falcon.falcon1a_decode_step(q, k, v, beta, lam, S.view(N * H, self.dim, self.dim),
                                        x_prev.view(N * H, self.dim))
        return o.view(N, H * self.dim) @ self.w_out.T

    def backward(self, kept, d_out):
        """Gradients of <d_out, out> of a fresh prompt, by parameter name."""
        r, rows, qkv, beta, lam, o = kept
        B, T = r.shape[:2]
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        d_o = (d_out @ self.w_out).view(B, T, self.heads, self.dim).transpose(1, 2).contiguous()
        g = falcon.falcon1a_bwd_chunked(*qkv, beta, lam, d_o)
        d_rows, d_w, d_b = torch.empty_like(rows), torch.empty_like(self.conv_w), \
            torch.empty_like(self.conv_b)
        for i, name in enumerate(("dq", "dk", "dv")):
            falcon.falcon_short_conv_bwd(
                self._heads(rows, i), self.conv_w[i], g[name], bias=self.conv_b[i],
                grads=dict(dx=self._heads(d_rows, i), dweight=d_w[i], dbias=d_b[i]))
        # through the sigmoid, and through softplus, whose slope is 1 - e^{-softplus}
        d_beta = (g["dbeta"] * beta * (1 - beta)).transpose(1, 2)
        d_lam = (g["dlambda"] * -torch.expm1(-lam)).transpose(1, 2)
        return dict(w_in=flat(d_rows).T @ flat(r), w_out=flat(d_out).T @ flat(o),
                    w_beta=flat(d_beta).T @ flat(r).float(), w_lam=flat(d_lam).T @ flat(r).float(),
                    conv_w=d_w, conv_b=d_b)


def train_step(layer, r, target, rate=100.0, max_norm=5e-3):
    """One step of gradient descent on the mean square error, gradients clipped."""
    out, _, kept = layer.prompt(r)
    off = out.float() - target.float()
    grads = layer.backward(kept, (off * (2.0 / off.numel())).to(layer.dtype))
    norm = falcon.falcon_clip_grad_norm(list(grads.values()), max_norm)
    for name, g in grads.items():
        p = getattr(layer, name)
        p.sub_((rate * g.float()).to(p.dtype))
    return off.square().mean(), norm


def main(width=512, heads=8, batch=4, tokens=1024, new=8, steps=4, dim=64, dtype=torch.bfloat16):
    torch.manual_seed(0)
    layer = FalconLayer(width, heads, dim, dtype=dtype)
    r = torch.randn(batch, tokens + new, width, device="cuda").to(dtype)
    want = layer.prompt(r)[0][:, tokens:].float()
    _, (tails, S, x_last), _ = layer.prompt(r[:, :tokens])
    got = torch.stack([layer.token(r[:, tokens + i], tails, S, x_last) for i in range(new)], 1)
    worst = float((got.float() - want).norm() / want.norm())
    print(f"{new} tokens after prompts of {tokens}: off by {worst:.1e} from longer prompts")
    target = torch.randn(batch, tokens, width, device="cuda").to(dtype)
    losses = []
    for i in range(steps):
        loss, norm = train_step(layer, r[:, :tokens], target)
        losses.append(float(loss))
        print(f"step {i}: loss {losses[-1]:.5f}, gradient norm {float(norm):.4f}")
    return worst, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    for name, value in (("width", 512), ("heads", 8), ("batch", 4), ("tokens", 1024), ("new", 8),
                        ("steps", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    main(**vars(ap.parse_args()))
