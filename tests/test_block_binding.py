"""The block's binding on the host: where its memory comes from and what it refuses, with
the library, the allocator and the streams replaced by recorders (no GPU needed)."""
import contextlib

import pytest
import torch

from delta_rule_attention_gb300 import block

F32, BF16 = torch.float32, torch.bfloat16


class OnGpu(torch.Tensor):
    """A host tensor that says it lies on a GPU."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    index = 0

    @property
    def device(self):
        return torch.device("cuda", self.index)

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        self.__dict__.setdefault("recorded", []).append(stream)


def _gpu(*shape, dtype=F32, index=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)
    t.index = index
    return t


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, torch.device("cuda", 0)


class World:
    """The current stream and device, what was allocated under which stream, and the
    library's calls."""

    def __init__(self, monkeypatch):
        self.here, self.device = Stream(0), 0
        self.now, self.allocated, self.calls = self.here, [], []

        @contextlib.contextmanager
        def on(stream):
            before, self.now = self.now, stream
            yield
            self.now = before

        def empty(shape, dtype=None, device=None):
            self.allocated.append(self.now)
            shape = (shape,) if isinstance(shape, int) else tuple(shape)
            return _gpu(*shape, dtype=dtype)

        def empty_like(t):
            return empty(t.shape, t.dtype)

        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch, "empty_like", empty_like)
        monkeypatch.setattr(block, "_new", empty)
        monkeypatch.setattr(block, "_raw_stream", lambda index: self.now.cuda_stream)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.device, raising=False)
        monkeypatch.setattr(block, "_device_now", lambda: self.device, raising=False)
        monkeypatch.setattr(torch.Tensor, "get_device", lambda t: getattr(t, "index", -1))
        monkeypatch.setattr(block, "_lib", self)

    def __getattr__(self, name):
        if not name.startswith("falcon"):
            raise AttributeError(name)

        def call(*args):
            if name.endswith("_bytes"):
                return 512
            self.calls.append((name, args))
            return 0

        return call


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def _calls():
    """Every entry point with arguments that it takes."""
    x, w, dy = _gpu(2, 5, 8), _gpu(8, 4), _gpu(2, 5, 8)
    A, bc, skip = _gpu(8, 16), _gpu(2, 5, 1, 16), _gpu(8)
    return {
        "short_conv_fwd": (block.falcon_short_conv_fwd, dict(x=x, weight=w)),
        "short_conv_bwd": (block.falcon_short_conv_bwd, dict(x=x, weight=w, dy=dy)),
        "short_conv_step": (block.falcon_short_conv_step,
                            dict(x=_gpu(2, 8), weight=w, state=_gpu(2, 3, 8))),
        "selective_scan_fwd": (block.falcon_selective_scan_fwd,
                               dict(u=x, delta=dy, A=A, Bm=bc, Cm=bc, D=skip, z=x)),
        "selective_scan_bwd": (block.falcon_selective_scan_bwd,
                               dict(u=x, delta=x, A=A, Bm=bc, Cm=bc, dy=dy, D=skip, z=x,
                                    delta_bias=skip)),
        "selective_scan_step": (block.falcon_selective_scan_step,
                                dict(u=_gpu(2, 8), delta=_gpu(2, 8), A=A, Bm=_gpu(2, 1, 16),
                                     Cm=_gpu(2, 1, 16), h=_gpu(2, 8, 16))),
        "clip_grad_norm": (block.falcon_clip_grad_norm,
                           dict(grads=[_gpu(8), _gpu(3, dtype=BF16)], max_norm=1.0)),
    }


def _tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    return [t for t in (out.values() if isinstance(out, dict) else out) if t is not None]


@pytest.mark.parametrize("name", sorted(_calls()))
def test_memory_of_a_call_on_a_given_stream_comes_from_that_stream(world, name):
    """Memory that the current stream's pool hands out may still be in use by work queued
    on it, which nothing orders before a call on another stream."""
    fn, args = _calls()[name]
    side = Stream(77)
    out = fn(**args, stream=side)
    assert world.allocated and all(s is side for s in world.allocated)
    (_, passed), = world.calls
    assert passed[-1] == 77
    assert world.now is world.here
    # the results are used, and may be dropped, on the current stream
    assert all(t.recorded == [world.here] for t in _tensors(out))


@pytest.mark.parametrize("name", sorted(_calls()))
def test_calls_on_the_current_stream_record_nothing(world, name):
    fn, args = _calls()[name]
    for out in (fn(**args), fn(**args, stream=world.here)):
        assert not any(hasattr(t, "recorded") for t in _tensors(out))
    assert all(s is world.here for s in world.allocated)
    assert [a[-1] for _, a in world.calls] == [0, 0]


def test_tensors_that_were_passed_in_are_not_recorded(world):
    x, w, y, tail = _gpu(2, 5, 8), _gpu(8, 4), _gpu(2, 5, 8), _gpu(2, 3, 8)
    out = block.falcon_short_conv_fwd(x, w, y=y, state_out=tail, stream=Stream(5))
    assert out[0] is y and out[1] is tail
    dx = _gpu(2, 5, 8)
    g = block.falcon_short_conv_bwd(x, w, x, grads={"dx": dx}, stream=Stream(5))
    assert g["dx"] is dx and g["dweight"].recorded == [world.here]
    assert not any(hasattr(t, "recorded") for t in (x, w, y, tail, dx))


@pytest.mark.parametrize("name", sorted(_calls()))
def test_tensors_on_a_gpu_that_is_not_the_current_one_are_refused(world, name):
    """A launch goes to the current device, whatever its pointers belong to."""
    fn, args = _calls()[name]
    world.device = 1
    with pytest.raises(ValueError, match="current"):
        fn(**args)
    assert world.calls == []
    world.device = 0
    fn(**args)
    assert len(world.calls) == 1


def test_the_fast_weight_calls_refuse_them_too(world, monkeypatch):
    import delta_rule_attention_gb300 as falcon
    monkeypatch.setattr(falcon, "_lib", world)
    world.device = 1
    q, beta = _gpu(2, 16), _gpu(2)
    with pytest.raises(ValueError, match="current"):
        falcon.falcon1_decode_step(q, q, q, beta, beta, _gpu(2, 16, 16), q)
    q, beta = _gpu(1, 1, 4, 16), _gpu(1, 1, 4)
    for call in (falcon.falcon1_fwd_chunked, falcon.falcon1a_fwd_chunked,
                 falcon.falcon2_fwd_recurrent, falcon.falcon1_fwd_chunked_fixed_scratch,
                 falcon.falcon1a_fwd_chunked_normalized):
        with pytest.raises(ValueError, match="current"):
            call(q, q, q, beta, beta)
    with pytest.raises(ValueError, match="current"):
        falcon.falcon1_bwd_chunked(q, q, q, beta, beta, q)
    assert world.calls == []


BAD_WORKSPACES = [(lambda: torch.zeros(4096, dtype=torch.uint8), ValueError),
                  (lambda: _gpu(4096, dtype=torch.uint8, index=1), ValueError),
                  (lambda: torch.zeros(64, 64)[:, ::2].as_subclass(OnGpu), ValueError),
                  (lambda: 4096, TypeError)]


@pytest.mark.parametrize("name", ["short_conv_bwd", "selective_scan_bwd", "clip_grad_norm"])
@pytest.mark.parametrize("make,error", BAD_WORKSPACES)
def test_workspaces_that_a_kernel_cannot_write_are_refused(world, name, make, error):
    fn, args = _calls()[name]
    with pytest.raises(error, match="workspace"):
        fn(**args, workspace=make())
    assert world.calls == []
    fn(**args, workspace=_gpu(1024))
    assert len(world.calls) == 1


@pytest.mark.parametrize("make,error", [
    (lambda: torch.zeros(()), ValueError), (lambda: _gpu(index=1), ValueError),
    (lambda: _gpu(dtype=torch.float64), TypeError), (lambda: _gpu(dtype=BF16), TypeError),
    (lambda: _gpu(0), ValueError), (lambda: _gpu(2), ValueError), (lambda: 0.0, TypeError)])
def test_a_norm_that_a_kernel_cannot_write_is_refused(world, make, error):
    fn, args = _calls()["clip_grad_norm"]
    with pytest.raises(error, match="norm"):
        fn(**args, norm=make())
    assert world.calls == []
    for norm in (_gpu(), _gpu(1)):
        assert fn(**args, norm=norm) is norm


def _fast_weight_calls():
    import delta_rule_attention_gb300 as f
    q, b, b2 = _gpu(1, 2, 4, 16), _gpu(1, 2, 4), _gpu(1, 2, 4, 16)
    n, nb = _gpu(2, 16), _gpu(2)
    return {
        "falcon1_fwd_chunked": (f.falcon1_fwd_chunked, (q, q, q, b, b), {}),
        "falcon1a_fwd_chunked": (f.falcon1a_fwd_chunked, (q, q, q, b, b), {}),
        "fixed_scratch": (f.falcon1_fwd_chunked_fixed_scratch, (q, q, q, b, b), {}),
        "normalized": (f.falcon1a_fwd_chunked_normalized, (q, q, q, b, b), {}),
        "falcon1_bwd_chunked": (f.falcon1_bwd_chunked, (q, q, q, b, b, q), {}),
        "falcon2_fwd_recurrent": (f.falcon2_fwd_recurrent, (q, q, q, b2, b), {}),
        "falcon2_fwd_chunked": (f.falcon2_fwd_chunked, (q, q, q, b2, b), {}),
        "falcon2a_fwd_chunked": (f.falcon2a_fwd_chunked, (q, q, q, b2, b), {}),
        "falcon3a_fwd_recurrent": (f.falcon3a_fwd_recurrent, (q, q, q, b, b), dict(window=4)),
        "falcon3a_fwd_chunked": (f.falcon3a_fwd_chunked, (q, q, q, b, b), dict(window=4)),
        "falcon1_decode_step": (f.falcon1_decode_step, (n, n, n, nb, nb, _gpu(2, 16, 16), n), {}),
    }


@pytest.mark.parametrize("name", sorted(_fast_weight_calls()))
def test_memory_of_a_fast_weight_call_on_a_given_stream_comes_from_it(world, monkeypatch, name):
    import delta_rule_attention_gb300 as falcon
    monkeypatch.setattr(falcon, "_lib", world)
    fn, args, kw = _fast_weight_calls()[name]
    side = Stream(77)
    out = fn(*args, **kw, stream=side)
    assert world.allocated and all(s is side for s in world.allocated)
    (_, passed), = world.calls
    assert passed[-1].value == 77
    assert all(t.recorded == [world.here] for t in _tensors(out))
    # on the current stream, nothing is recorded
    for out in (fn(*args, **kw), fn(*args, **kw, stream=world.here)):
        assert not any(hasattr(t, "recorded") for t in _tensors(out))


def test_a_fast_weight_call_keeps_its_options_on_a_given_stream(world, monkeypatch):
    """The library gets the same arguments whichever way the stream is named."""
    import delta_rule_attention_gb300 as falcon
    monkeypatch.setattr(falcon, "_lib", world)
    q, b = _gpu(1, 2, 4, 16), _gpu(1, 2, 4)
    o, S, xl, ws = _gpu(1, 2, 4, 16), _gpu(1, 2, 16, 16), _gpu(1, 2, 16), _gpu(4096)
    S0, xp, z0 = _gpu(1, 2, 16, 16), _gpu(1, 2, 16), _gpu(1, 2, 16)
    opts = dict(phi="rms", eps=1e-3, eps_gamma=1e-4, ridge="scaled")
    n, nb = _gpu(2, 16), _gpu(2)
    fresh = _gpu(2, dtype=torch.uint8)
    dS, dx = _gpu(1, 2, 16, 16), _gpu(1, 2, 16)
    g = {k: _gpu(1, 2, 4, 16) for k in ("dq", "dk", "dv")}
    g.update(dbeta=_gpu(1, 2, 4), dlambda=_gpu(1, 2, 4), dS0=_gpu(1, 2, 16, 16),
             dx_prev=_gpu(1, 2, 16))
    outs = dict(o=o, S_out=S, x_last=xl)
    calls = [
        (falcon.falcon1_fwd_chunked, (q, q, q, b, b, S0, xp, 32),
         dict(outs, workspace=ws, **opts)),
        (falcon.falcon1_fwd_chunked_fixed_scratch, (q, q, q, b, b, S0, xp, 32), dict(outs, **opts)),
        (falcon.falcon1a_fwd_chunked_normalized, (q, q, q, b, b, S0, z0, xp, 1e-2, 32),
         dict(outs, z_out=_gpu(1, 2, 16), workspace=ws, **opts)),
        (falcon.falcon1a_bwd_chunked, (q, q, q, b, b, q, S0, xp, dS, dx, 32),
         dict(workspace=ws, grads=g, **opts)),
        (falcon.falcon2a_fwd_chunked, (q, q, q, _gpu(1, 2, 4, 16), b, S0, xp),
         dict(outs, workspace=ws, **opts)),
        (falcon.falcon2_fwd_recurrent, (q, q, q, _gpu(1, 2, 4, 16), b, S0, xp), dict(outs, **opts)),
        (falcon.falcon3a_fwd_recurrent, (q, q, q, b, b, 5, S0), dict(outs, **opts)),
        (falcon.falcon3a_fwd_chunked, (q, q, q, b, b, 5, S0), dict(outs, workspace=ws, **opts)),
        (falcon.falcon1a_decode_step, (n, n, n, nb, nb, _gpu(2, 16, 16), n, fresh),
         dict(o=_gpu(2, 16), **opts)),
    ]

    def plain(a):
        if hasattr(a, "_obj"):  # a reference to a structure
            return bytes(a._obj)
        return getattr(a, "value", a)

    for fn, args, kw in calls:
        world.calls.clear()
        fn(*args, **kw)
        fn(*args, **kw, stream=Stream(9))
        (n0, a), (n1, c) = world.calls
        assert n0 == n1 and plain(c[-1]) == 9
        assert [plain(v) for v in a[:-1]] == [plain(v) for v in c[:-1]], fn
