"""Scans whose decay rates reach the ends of float32 (A = -3e38 and -inf): a step of zero
leaves the state, any other erases it, and what lies behind a row's length plays no
part.  The reference takes an infinite rate as the largest float32, as the library says.

Tolerances as in test_gpu_block.py: (T + 16) 2^-21, plus 2^-8 for a stored bf16."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def falcon():
    import delta_rule_attention_gb300 as m
    return m


def _case(dtype, B, T, D, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    A = -torch.exp(r(D, N))
    A[0], A[1, ::2], A[2], A[3, 1::2] = -3e38, -2.5e38, float("-inf"), float("-inf")
    return dict(u=r(B, T, D).to(dtype), delta=(0.5 * r(B, T, D)).to(dtype), A=A,
                Bm=r(B, T, 1, N).to(dtype), Cm=r(B, T, 1, N).to(dtype), D=r(D),
                h0=r(B, D, N))


def _reference(d):
    r = {k: v if k == "lengths" else ref.f64(v) for k, v in d.items()}
    r["A"] = r["A"].clamp(min=torch.finfo(F32).min)
    return r


def _tol(dtype, T):
    return (T + 16) * 2.0 ** -21 + (2.0 ** -8 if dtype == BF16 else 0.0)


def _check(got, want, tol, name):
    assert bool(got.isfinite().all()), name
    assert ref.rel(got, want) <= tol, (name, ref.rel(got, want))


@pytest.mark.parametrize("T,D,N", [(21, 16, 16), (21, 7, 5), (1301, 16, 16), (600, 8, 33)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_and_gradient_of_ragged_rows(dtype, T, D, N):
    d = _case(dtype, 4, T, D, N)
    d["lengths"] = torch.tensor([T, 0, T // 2 + 1, 1], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    dy, dh = torch.randn(4, T, D, generator=g).to(dtype), torch.randn(4, D, N, generator=g)
    c = {k: v.cuda() for k, v in d.items()}
    m = falcon()
    y, h = m.falcon_selective_scan_fwd(**c)
    got = m.falcon_selective_scan_bwd(**c, dy=dy.cuda(), dh_T=dh.cuda())
    r = _reference(d)
    wy, wh = ref.scan(**r)
    _check(y, wy, _tol(dtype, T), "y")
    _check(h, wh, _tol(F32, T), "h")
    want = ref.gradients(ref.scan, r, [ref.f64(dy), ref.f64(dh)])
    for mine, theirs in (("du", "u"), ("ddelta", "delta"), ("dB", "Bm"), ("dC", "Cm"), ("dA", "A"),
                         ("dD", "D"), ("dh0", "h0")):
        dt = dtype if mine in ("du", "ddelta", "dB", "dC") else F32
        _check(got[mine], want[theirs], _tol(dt, T), mine)


@pytest.mark.parametrize("D,N", [(16, 16), (7, 5)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_steps_of_zero_leave_the_state(dtype, D, N):
    d = _case(dtype, 3, 9, D, N)
    d["delta"][:, 2], d["delta"][:, 5:7], d["delta"][1] = -300.0, float("-inf"), float("-inf")
    m, r = falcon(), _reference(d)
    r["delta"] = r["delta"].clamp(min=-1e4)  # softplus(-1e4) is zero in float64 too
    y, h = m.falcon_selective_scan_fwd(**{k: v.cuda() for k, v in d.items()})
    wy, wh = ref.scan(**r)
    _check(y, wy, _tol(dtype, 9), "y")
    _check(h, wh, _tol(F32, 9), "h")
    pool = d["h0"].cuda()
    one = {k: d[k][:, 2].cuda() for k in ("u", "delta", "Bm", "Cm")}
    m.falcon_selective_scan_step(one["u"], one["delta"], d["A"].cuda(), one["Bm"], one["Cm"], pool,
                                 D=d["D"].cuda())
    assert torch.equal(pool.cpu(), d["h0"])
