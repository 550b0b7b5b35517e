"""A linear attention model with a fixed decay for each head: a prompt, the tokens after it,
and training steps with the gradients clipped.

    python examples/decay_block.py [--width 512] [--heads 8] [--layers 2] [--batch 4] [--tokens 1024]

A block is  q, k, v, z = W_in u,  o = decay attention(q, k, v),  y = norm(o by heads) w
silu(z),  h = W_out y,  x = x + s norm(h) w',  and the next block's u = norm(x) w''.  The
attention reads q, k and v from the projection's rows; the norm behind it turns the
heads back into rows and gates them; the norm behind the block adds the residual and
normalises it for the next block, each in one pass.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import delta_rule_attention_gb300 as falcon  # noqa: E402


class DecayModel:
    """Parameters of `layers` blocks with `heads` heads of `dim` keys and values each."""

    def __init__(self, width, heads, layers=2, dim=64, dtype=torch.bfloat16, device="cuda",
                 seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        channels = heads * dim

        def mat(out, inn):
            return (torch.randn(out, inn, generator=g, device=device) * inn ** -0.5).to(dtype)

        def near(n, value):
            return value + 0.05 * torch.randn(n, generator=g, device=device)

        self.heads, self.dim, self.layers, self.dtype = heads, dim, layers, dtype
        # half-lives of about 2 to 700 tokens
        self.log_decay = -torch.exp2(-1.5 - 8.5 * torch.arange(heads, device=device)
                                     / max(heads - 1, 1))
        self.norm_in = near(width, 1.0)
        self.blocks = [dict(w_in=mat(4 * channels, width), w_out=mat(width, channels),
                            norm_heads=near(channels, 1.0), norm_post=near(width, 1.0),
                            scale=near(width, 0.5), norm_next=near(width, 1.0))
                       for _ in range(layers)]

    def parts(self, rows):
        """q, k, v [B,H,T,dim] and the gate's rows [B,T,H*dim]: views of [B,T,4*H*dim]."""
        B, T = rows.shape[:2]
        qkv = rows[..., :3 * self.heads * self.dim].unflatten(2, (3, self.heads, self.dim))
        q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
        return q, k, v, rows[..., 3 * self.heads * self.dim:]

    def prompt(self, x, states=None, lengths=None):
        """x [B,T,width] -> (out, states, what the gradient needs)."""
        _, u = falcon.falcon_gated_norm_fwd(None, x=x, next_weight=self.norm_in, lengths=lengths)
        ends, kept = [], [x]
        for i, p in enumerate(self.blocks):
            rows = u @ p["w_in"].T
            q, k, v, z = self.parts(rows)
            o, S = falcon.falcon_decay_attn_fwd(q, k, v, self.log_decay, lengths=lengths,
                                                S0=None if states is None else states[i])
            y, _ = falcon.falcon_gated_norm_fwd(o, weight=p["norm_heads"], z=z, lengths=lengths)
            h = y @ p["w_out"].T
            x, after = falcon.falcon_gated_norm_fwd(
                h, weight=p["norm_post"], scale=p["scale"], x=x, next_weight=p["norm_next"],
                lengths=lengths)
            kept.append((u, rows, o, y, h, x))
            ends.append(S)
            u = after
        return u, ends, (kept, lengths)

    def token(self, x, states, slots=None):
        """x [N,width], one token of N sequences; their states are updated in place."""
        x = x[:, None]
        _, u = falcon.falcon_gated_norm_fwd(None, x=x, next_weight=self.norm_in)
        for p, S in zip(self.blocks, states):
            q, k, v, z = self.parts(u @ p["w_in"].T)
            o = falcon.falcon_decay_attn_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], self.log_decay,
                                              S, slots=slots)
            y, _ = falcon.falcon_gated_norm_fwd(o[:, :, None], weight=p["norm_heads"], z=z)
            x, u = falcon.falcon_gated_norm_fwd(
                y @ p["w_out"].T, weight=p["norm_post"], scale=p["scale"], x=x,
                next_weight=p["norm_next"])
        return u[:, 0]

    def backward(self, kept, d_out):
        """Gradients of <d_out, out> of a fresh prompt: (the model's, a dict a block, x's)."""
        (x0, *blocks), lengths = kept
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        grads, d_x, d_u = [None] * self.layers, None, d_out
        for i in reversed(range(self.layers)):
            p, (u, rows, o, y, h, x) = self.blocks[i], blocks[i]
            q, k, v, z = self.parts(rows)
            post = falcon.falcon_gated_norm_bwd(
                h, d_x, dnext=d_u, out=x, weight=p["norm_post"], scale=p["scale"],
                next_weight=p["norm_next"], lengths=lengths)
            d_x, d_h = post["dx"], post["dh"]
            d_rows = torch.empty_like(rows)
            d_q, d_k, d_v, d_z = self.parts(d_rows)
            gate = falcon.falcon_gated_norm_bwd(
                o, d_h @ p["w_out"], weight=p["norm_heads"], z=z, residual=False,
                lengths=lengths, grads=dict(dz=d_z))
            falcon.falcon_decay_attn_bwd(q, k, v, self.log_decay, gate["dh"], lengths=lengths,
                                         grads=dict(dq=d_q, dk=d_k, dv=d_v))
            grads[i] = dict(w_in=flat(d_rows).T @ flat(u), w_out=flat(d_h).T @ flat(y),
                            norm_heads=gate["dweight"], norm_post=post["dweight"],
                            scale=post["dscale"], norm_next=post["dnext_weight"])
            d_u = d_rows @ p["w_in"]
        first = falcon.falcon_gated_norm_bwd(None, d_x, dnext=d_u, out=x0,
                                             next_weight=self.norm_in, lengths=lengths)
        return dict(norm_in=first["dnext_weight"]), grads, first["dx"]


def train_step(model, x, target, rate=50.0, max_norm=5e-3):
    """One step of gradient descent on the mean square error, gradients clipped."""
    out, _, kept = model.prompt(x)
    off = out.float() - target.float()
    own, blocks, _ = model.backward(kept, (off * (2.0 / off.numel())).to(model.dtype))
    flat = list(own.values()) + [g for b in blocks for g in b.values()]
    norm = falcon.falcon_clip_grad_norm(flat, max_norm)
    params = [model.norm_in] + [p[n] for p, b in zip(model.blocks, blocks) for n in b]
    for p, g in zip(params, flat):
        p.sub_((rate * g.float()).to(p.dtype))
    return off.square().mean(), norm


def main(width=512, heads=8, layers=2, batch=4, tokens=1024, new=8, steps=4, dim=64,
         dtype=torch.bfloat16):
    torch.manual_seed(0)
    model = DecayModel(width, heads, layers, dim, dtype=dtype)
    x = torch.randn(batch, tokens + new, width, device="cuda").to(dtype)
    want = model.prompt(x)[0][:, tokens:].float()
    _, states, _ = model.prompt(x[:, :tokens])
    got = torch.stack([model.token(x[:, tokens + i], states) for i in range(new)], 1)
    worst = float((got.float() - want).norm() / want.norm())
    print(f"{new} tokens after prompts of {tokens}: off by {worst:.1e} from longer prompts")
    target = torch.randn(batch, tokens, width, device="cuda").to(dtype)
    losses = []
    for i in range(steps):
        loss, norm = train_step(model, x[:, :tokens], target)
        losses.append(float(loss))
        print(f"step {i}: loss {losses[-1]:.5f}, gradient norm {float(norm):.4f}")
    return worst, losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    for name, value in (("width", 512), ("heads", 8), ("layers", 2), ("batch", 4),
                        ("tokens", 1024), ("new", 8), ("steps", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    main(**vars(ap.parse_args()))
