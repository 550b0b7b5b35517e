"""The linear attention block's binding on the host: where its memory comes from and what it
refuses, with the library, the allocator and the streams replaced by recorders (no GPU)."""
import pytest
import torch

from delta_rule_attention_gb300 import block, linear
from test_block_binding import BF16, F32, Stream, World, _gpu


@pytest.fixture
def world(monkeypatch):
    for f in ("_decay_shape", "_norm_shape", "_need"):
        getattr(linear, f).cache_clear()
    w = World(monkeypatch)
    yield w
    linear._need.cache_clear()


def fwd(**kw):
    a = dict(q=_gpu(2, 3, 4, 8), k=_gpu(2, 3, 4, 8), v=_gpu(2, 3, 4, 6), log_decay=_gpu(3))
    a.update(kw)
    return linear.falcon_decay_attn_fwd(**a)


def bwd(**kw):
    a = dict(q=_gpu(2, 3, 4, 8), k=_gpu(2, 3, 4, 8), v=_gpu(2, 3, 4, 6), log_decay=_gpu(3),
             dO=_gpu(2, 3, 4, 6))
    a.update(kw)
    return linear.falcon_decay_attn_bwd(**a)


def step(**kw):
    a = dict(q=_gpu(2, 3, 8), k=_gpu(2, 3, 8), v=_gpu(2, 3, 6), log_decay=_gpu(3),
             S=_gpu(2, 3, 8, 6))
    a.update(kw)
    return linear.falcon_decay_attn_step(**a)


def norm(**kw):
    a = dict(h=_gpu(2, 3, 4, 8), weight=_gpu(24), z=_gpu(2, 4, 24), x=_gpu(2, 4, 24),
             next_weight=_gpu(24))
    a.update(kw)
    return linear.falcon_gated_norm_fwd(**a)


def norm_bwd(**kw):
    a = dict(h=_gpu(2, 3, 4, 8), dout=_gpu(2, 4, 24), dnext=_gpu(2, 4, 24), out=_gpu(2, 4, 24),
             weight=_gpu(24), z=_gpu(2, 4, 24), next_weight=_gpu(24))
    a.update(kw)
    return linear.falcon_gated_norm_bwd(**a)


CALLS = (fwd, bwd, step, norm, norm_bwd)


@pytest.mark.parametrize("call", CALLS)
def test_a_call_allocates_under_the_stream_it_is_given(world, call):
    call()
    assert world.allocated and all(s is world.here for s in world.allocated)
    world.allocated.clear()
    other = Stream(7)
    out = call(stream=other)
    assert world.allocated and all(s is other for s in world.allocated)
    new = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)
    for t in new:
        assert t is None or t.__dict__.get("recorded") == [world.here]


@pytest.mark.parametrize("call", CALLS)
def test_another_device_is_refused(world, call):
    world.device = 1
    with pytest.raises(ValueError, match="current device"):
        call()


@pytest.mark.parametrize("bad", [
    dict(q=_gpu(2, 3, 4, 8, dtype=torch.float16)), dict(q=torch.zeros(2, 3, 4, 8)),
    dict(q=_gpu(2, 3, 32)), dict(k=_gpu(2, 3, 4, 7)), dict(k=_gpu(2, 3, 4, 8, dtype=BF16)),
    dict(v=_gpu(2, 3, 5, 6)), dict(v=_gpu(2, 3, 4)), dict(v=_gpu(2, 3, 4, 6, index=1)),
    dict(log_decay=_gpu(2)), dict(log_decay=_gpu(3, dtype=BF16)), dict(log_decay=None),
    dict(S0=_gpu(2, 3, 6, 8)), dict(lengths=_gpu(2, dtype=torch.int64)),
    dict(lengths=_gpu(3, dtype=torch.int32)), dict(o=_gpu(2, 3, 4, 8)),
    dict(S_out=_gpu(2, 3, 8, 6, dtype=BF16)), dict(workspace=torch.zeros(4)),
    dict(q=_gpu(2, 3, 8, 4).transpose(2, 3)),
])
def test_decay_forward_refuses(world, bad):
    with pytest.raises((TypeError, ValueError)):
        fwd(**bad)


@pytest.mark.parametrize("bad", [
    dict(dO=_gpu(2, 3, 4, 8)), dict(dO=None), dict(dS_T=_gpu(2, 3, 8)),
    dict(grads=dict(dq=_gpu(2, 3, 4, 6))), dict(grads=dict(dS0=_gpu(2, 3, 8, 6, dtype=BF16))),
])
def test_decay_backward_refuses(world, bad):
    with pytest.raises((TypeError, ValueError)):
        bwd(**bad)


@pytest.mark.parametrize("bad", [
    dict(S=_gpu(3, 3, 8, 6)), dict(S=_gpu(2, 3, 48)), dict(S=_gpu(2, 3, 8, 6, dtype=BF16)),
    dict(slots=_gpu(2, dtype=torch.int64)), dict(fresh=_gpu(2)), dict(o=_gpu(2, 3, 8)),
    dict(k=_gpu(2, 3, 7)), dict(q=_gpu(2, 24)),
])
def test_decay_step_refuses(world, bad):
    with pytest.raises((TypeError, ValueError)):
        step(**bad)


@pytest.mark.parametrize("bad", [
    dict(h=_gpu(2, 24)), dict(weight=_gpu(8)), dict(weight=_gpu(24, dtype=BF16)),
    dict(z=_gpu(2, 3, 4, 8)), dict(x=_gpu(2, 4, 24, dtype=BF16)), dict(gate="tanh"),
    dict(next_weight=None, next_out=_gpu(2, 4, 24)), dict(h=None), dict(out=_gpu(2, 4, 8)),
    dict(lengths=_gpu(2)), dict(h=None, weight=None, z=None, next_weight=None),
])
def test_norm_forward_refuses(world, bad):
    with pytest.raises((TypeError, ValueError)):
        norm(**bad)


@pytest.mark.parametrize("bad", [
    dict(dnext=None), dict(out=None), dict(next_weight=None), dict(h=None),
    dict(dout=None, dnext=None, next_weight=None), dict(dout=_gpu(2, 3, 4, 8)),
    dict(grads=dict(dh=_gpu(2, 4, 24))), dict(grads=dict(dweight=_gpu(8))),
])
def test_norm_backward_refuses(world, bad):
    with pytest.raises((TypeError, ValueError)):
        norm_bwd(**bad)


def test_results_of_what_was_not_given(world):
    g = norm_bwd(z=None, residual=False, scale=None)
    assert g["dz"] is None and g["dx"] is None and g["dscale"] is None
    assert g["dh"].shape == (2, 3, 4, 8) and g["dnext_weight"].shape == (24,)
    out, nxt = norm(next_weight=None, x=None, z=None, weight=None)
    assert nxt is None and out.shape == (2, 4, 24)
    x = _gpu(2, 4, 24)
    out, nxt = norm(h=None, weight=None, z=None, x=x)
    assert out is x and nxt.shape == (2, 4, 24)


@pytest.mark.parametrize("name,without", [
    ("dx", dict(residual=False)), ("dz", dict(z=None)), ("dweight", dict(weight=None)),
    ("dscale", dict(scale=None)),
    ("dnext_weight", dict(next_weight=None, dnext=None)),
    ("dh", dict(h=None, weight=None, z=None)),
])
def test_a_result_of_what_was_not_given_is_refused(world, name, without):
    """It would be left as it is; the caller's dict keeps it."""
    t = _gpu(2, 3, 4, 8) if name == "dh" else _gpu(2, 4, 24) if name in ("dx", "dz") else _gpu(24)
    grads = {name: t}
    with pytest.raises(ValueError, match=name):
        norm_bwd(grads=grads, **without)
    assert grads == {name: t} and not world.calls


def test_results_of_a_call_are_passed_to_the_next(world):
    """With the None of what was not given, which stays, or is allocated where it is now."""
    g = norm_bwd(z=None, scale=None)
    assert g["dz"] is None
    kept = {n: t for n, t in g.items() if t is not None}
    assert norm_bwd(z=None, scale=None, grads=g) is g
    assert all(g[n] is t for n, t in kept.items())
    norm_bwd(grads=g)
    assert g["dz"].shape == (2, 4, 24) and all(g[n] is t for n, t in kept.items())


def test_keys_of_no_channel_are_refused_by_the_library(world):
    """Not by a division of one by zero on the way there."""
    wide = dict(q=_gpu(2, 3, 4, 0), k=_gpu(2, 3, 4, 0))
    fwd(**wide)
    bwd(**wide)
    step(q=_gpu(2, 3, 0), k=_gpu(2, 3, 0), S=_gpu(2, 3, 0, 6))
    assert [name for name, _ in world.calls] == [
        "falcon_decay_attn_fwd", "falcon_decay_attn_bwd", "falcon_decay_attn_step"]
