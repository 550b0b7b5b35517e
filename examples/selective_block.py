"""A selective state space block over the library's entry points: a prompt, the
tokens after it, and one training step with its gradients clipped.

    python examples/selective_block.py [--width 512] [--batch 8] [--tokens 1024]

The block is  x, z = split(W_in r);  x = silu(conv(x));  delta, B, C = split(W_x x);
delta = W_dt delta;  y = scan(x, delta, A, B, C, D, z);  out = W_out y.  Its matrix
products are plain library products; everything between them is this library's.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import delta_rule_attention_gb300 as falcon  # noqa: E402


class SelectiveBlock:
    """Parameters of one block; ``inner`` = 2 width channels, ``states`` a channel."""

    def __init__(self, width, states=16, taps=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def mat(out, inn):
            return (torch.randn(out, inn, generator=g, device=device) * inn ** -0.5).to(dtype)

        inner, rank = 2 * width, max(8, width // 8)
        self.inner, self.rank, self.states, self.taps, self.dtype = inner, rank, states, taps, dtype
        self.w_in, self.w_out = mat(2 * inner, width), mat(width, inner)
        self.w_x, self.w_dt = mat(rank + 2 * states, inner), mat(inner, rank)
        self.conv_w = torch.randn(inner, taps, generator=g, device=device) * taps ** -0.5
        self.conv_b = torch.zeros(inner, device=device)
        self.A = -torch.arange(1, states + 1, device=device).float().repeat(inner, 1)
        steps = torch.exp(torch.rand(inner, generator=g, device=device) * math.log(100.0)
                          + math.log(1e-3))
        self.dt_bias = steps + torch.log(-torch.expm1(-steps))
        self.D = torch.ones(inner, device=device)

    def _scan_inputs(self, x):
        rank, n = self.rank, self.states
        p = x @ self.w_x.T
        groups = p.shape[:-1] + (1, n)
        return (p[..., :rank], p[..., rank:rank + n].view(groups), p[..., rank + n:].view(groups))

    def prompt(self, r, lengths=None, conv_state=None, h=None):
        """r [B,T,width] -> (out, conv_state, h, kept for backward)."""
        xz = r @ self.w_in.T
        x0, z = xz[..., :self.inner], xz[..., self.inner:]
        x, tail = falcon.falcon_short_conv_fwd(x0, self.conv_w, bias=self.conv_b,
                                               state=conv_state, lengths=lengths)
        low, B, C = self._scan_inputs(x)
        delta = low @ self.w_dt.T
        y, h_T = falcon.falcon_selective_scan_fwd(x, delta, self.A, B, C, D=self.D, z=z,
                                                  delta_bias=self.dt_bias, h0=h, lengths=lengths)
        return y @ self.w_out.T, tail, h_T, (r, x0, z, x, low, B, C, delta, y)

    def token(self, r, conv_states, states, slots=None):
        """r [N,width], one token of N sequences whose states lie in pools."""
        xz = r @ self.w_in.T
        x = falcon.falcon_short_conv_step(xz[:, :self.inner], self.conv_w, conv_states,
                                          bias=self.conv_b, slots=slots)
        low, B, C = self._scan_inputs(x)
        y = falcon.falcon_selective_scan_step(x, low @ self.w_dt.T, self.A, B, C, states,
                                              D=self.D, z=xz[:, self.inner:],
                                              delta_bias=self.dt_bias, slots=slots)
        return y @ self.w_out.T

    def backward(self, kept, d_out):
        """Gradients of <d_out, out> of a fresh prompt, by parameter name."""
        r, x0, z, x, low, B, C, delta, y = kept
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        g = falcon.falcon_selective_scan_bwd(x, delta, self.A, B, C, d_out @ self.w_out, D=self.D,
                                             z=z, delta_bias=self.dt_bias)
        d_low = g["ddelta"] @ self.w_dt
        d_p = torch.cat([d_low, g["dB"].flatten(2), g["dC"].flatten(2)], -1)
        c = falcon.falcon_short_conv_bwd(x0, self.conv_w, g["du"] + d_p @ self.w_x,
                                         bias=self.conv_b)
        d_xz = torch.cat([c["dx"], g["dz"]], -1)
        return dict(w_out=flat(d_out).T @ flat(y), w_dt=flat(g["ddelta"]).T @ flat(low),
                    w_x=flat(d_p).T @ flat(x), w_in=flat(d_xz).T @ flat(r), A=g["dA"], D=g["dD"],
                    dt_bias=g["ddelta_bias"], conv_w=c["dweight"], conv_b=c["dbias"])


def train_step(block, r, target, rate=0.1, max_norm=1.0):
    """One step of gradient descent on the mean square error, gradients clipped."""
    out, _, _, kept = block.prompt(r)
    off = out.float() - target.float()
    d_out = (off * (2.0 / off.numel())).to(block.dtype)
    grads = block.backward(kept, d_out)
    norm = falcon.falcon_clip_grad_norm(list(grads.values()), max_norm)
    for name, g in grads.items():
        getattr(block, name).sub_((rate * g.float()).to(getattr(block, name).dtype))
    return off.square().mean(), norm


def main(width=512, batch=8, tokens=1024, new=8, steps=4):
    torch.manual_seed(0)
    block = SelectiveBlock(width)
    r = torch.randn(batch, tokens + new, width, device="cuda").to(block.dtype)
    # prompts of uneven lengths, then `new` tokens for all of them
    lengths = torch.randint(1, tokens + 1, (batch,), device="cuda", dtype=torch.int32)
    _, conv_state, h, _ = block.prompt(r[:, :tokens], lengths=lengths)
    rows = [block.token(r[:, tokens + i], conv_state, h) for i in range(new)]
    # the same rows as prompts that end with those tokens
    worst = 0.0
    for b in range(batch):
        n = int(lengths[b])
        whole = torch.cat([r[b, :n], r[b, tokens:]])[None]
        want = block.prompt(whole)[0][0, n:].float()
        got = torch.stack([row[b] for row in rows]).float()
        worst = max(worst, float((got - want).norm() / want.norm()))
    print(f"{new} tokens after prompts of {lengths.tolist()}: off by {worst:.1e} from longer prompts")
    target = torch.randn(batch, tokens, width, device="cuda").to(block.dtype)
    losses = []
    for i in range(steps):
        loss, norm = train_step(block, r[:, :tokens], target)
        losses.append(float(loss))
        print(f"step {i}: loss {losses[-1]:.5f}, gradient norm {float(norm):.4f}")
    return worst, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    for name, value in (("width", 512), ("batch", 8), ("tokens", 1024), ("new", 8), ("steps", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    main(**vars(ap.parse_args()))
