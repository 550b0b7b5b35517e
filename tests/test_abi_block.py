"""Argument checks of the selective state space block's entry points: refused
before a device is touched, with nothing launched (no GPU needed)."""
import ctypes
import os
import shutil

import pytest
import torch

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")

BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from delta_rule_attention_gb300 import _build
    _build.build()
    import delta_rule_attention_gb300 as falcon
    return falcon.load_library()


def _p(addr=0x10000):
    return ctypes.c_void_p(addr)


def _strides(batch=1024, head=0, time=16):
    from delta_rule_attention_gb300.block import falcon_strides
    return falcon_strides(batch, head, time)


def _conv_shape(**kw):
    from delta_rule_attention_gb300.block import falcon_conv_shape
    base = dict(B=2, H=1, T=8, m=16, width=4, dtype=F32, activation=1)
    base.update(kw)
    return falcon_conv_shape(*[base[f] for f, _ in falcon_conv_shape._fields_])


def _scan_shape(**kw):
    from delta_rule_attention_gb300.block import falcon_scan_shape
    base = dict(B=2, T=8, D=16, G=2, N=16, dtype=F32, softplus=1)
    base.update(kw)
    return falcon_scan_shape(*[base[f] for f, _ in falcon_scan_shape._fields_])


BAD_CONV = [(dict(B=-1), -2), (dict(T=-1), -2), (dict(m=0), -2), (dict(width=1), -2),
            (dict(width=5), -2), (dict(H=1 << 40), -2), (dict(dtype=2), -3),
            (dict(activation=2), -8)]


def _conv_fwd(lib, s, x=_p(), xs=None, w=_p(), bias=None, state=None, lengths=None, y=_p(),
              ys=None, out=None):
    return lib.falcon_short_conv_fwd(s, x, xs or _strides(), w, bias, state, lengths, y,
                                     ys or _strides(), out, None)


@pytest.mark.parametrize("bad,code", BAD_CONV)
def test_conv_forward_refuses_bad_shapes(lib, bad, code):
    assert _conv_fwd(lib, _conv_shape(**bad)) == code


def test_conv_forward_refuses_bad_pointers(lib):
    s = _conv_shape()
    assert _conv_fwd(lib, None) == -1
    assert _conv_fwd(lib, s, x=None) == -1
    assert _conv_fwd(lib, s, y=None) == -1
    assert _conv_fwd(lib, s, w=None) == -1
    assert _conv_fwd(lib, s, x=_p(0x10002)) == -4
    assert _conv_fwd(lib, s, lengths=_p(0x10002)) == -4
    assert _conv_fwd(lib, _conv_shape(dtype=BF16), x=_p(0x10001)) == -4
    assert _conv_fwd(lib, s, xs=_strides(time=-16)) == -8
    assert _conv_fwd(lib, s, state=_p(0x20000), out=_p(0x20000)) == -8
    assert _conv_fwd(lib, _conv_shape(B=0), x=None, w=None, y=None) == 0


def _conv_bwd(lib, s, x=_p(), dy=_p(), dx=_p(), dw=_p(), dstate=None, dso=None, ws=_p(),
              have=1 << 40, dys=None):
    return lib.falcon_short_conv_bwd(s, x, _strides(), _p(), None, None, None, dy,
                                     dys or _strides(), dso, dx, _strides(), dw, None, dstate, ws,
                                     have, None)


@pytest.mark.parametrize("bad,code", BAD_CONV)
def test_conv_backward_refuses_bad_shapes(lib, bad, code):
    assert _conv_bwd(lib, _conv_shape(**bad)) == code
    assert lib.falcon_short_conv_bwd_workspace_bytes(_conv_shape(**bad)) == 0


def test_conv_backward_refuses_bad_pointers_and_workspaces(lib):
    s = _conv_shape()
    assert lib.falcon_short_conv_bwd_workspace_bytes(s) > 0
    assert _conv_bwd(lib, s, x=None) == -1
    assert _conv_bwd(lib, s, dy=None) == -1
    assert _conv_bwd(lib, s, dx=None) == -1
    assert _conv_bwd(lib, s, dw=None) == -1
    assert _conv_bwd(lib, s, dx=_p(0x10002)) == -4
    assert _conv_bwd(lib, s, ws=_p(0x10008)) == -4
    assert _conv_bwd(lib, s, ws=None) == -5
    assert _conv_bwd(lib, s, have=4) == -5
    assert _conv_bwd(lib, s, dys=_strides(batch=-1)) == -8
    assert _conv_bwd(lib, s, dstate=_p(0x20000), dso=_p(0x20000)) == -8


def test_conv_step_refuses(lib):
    def step(N=2, C=16, W=4, dt=F32, act=1, x=_p(), xs=16, w=_p(), st=_p(), pool=2, y=_p(),
             slots=None):
        return lib.falcon_short_conv_step(N, C, W, dt, act, x, xs, w, None, st, pool, slots, None,
                                          y, None)
    assert step(N=-1) == -2
    assert step(W=1) == -2
    assert step(pool=-1) == -2
    assert step(N=1 << 40) == -2
    assert step(dt=9) == -3
    assert step(act=3) == -8
    assert step(xs=-1) == -8
    assert step(x=None) == -1
    assert step(st=None) == -1
    assert step(y=_p(0x10002)) == -4
    assert step(slots=_p(0x10001)) == -4
    assert step(N=0, x=None) == 0


BAD_SCAN = [(dict(B=-1), -2), (dict(T=-1), -2), (dict(G=0), -2), (dict(G=3), -2), (dict(N=0), -2),
            (dict(N=129), -2), (dict(B=65536), -2), (dict(dtype=2), -3)]


def _scan_fwd(lib, s, u=_p(), us=None, A=_p(), z=None, zs=None, y=_p(), h=_p(), bs=None):
    st = _strides()
    return lib.falcon_selective_scan_fwd(s, u, us or st, _p(), st, A, _p(), bs or st, _p(), st,
                                         None, z, zs, None, None, None, y, st, h, None)


def _scan_bwd(lib, s, u=_p(), dy=_p(), dA=_p(), z=None, dz=None, ws=_p(), have=1 << 50):
    st = _strides()
    return lib.falcon_selective_scan_bwd(s, u, st, _p(), st, _p(), _p(), st, _p(), st, None, z,
                                         st, None, None, None, dy, st, None, _p(), _p(), dA, _p(),
                                         _p(), None, dz, None, None, ws, have, None)


@pytest.mark.parametrize("bad,code", BAD_SCAN)
def test_scan_refuses_bad_shapes(lib, bad, code):
    s = _scan_shape(**bad)
    assert _scan_fwd(lib, s) == code
    assert _scan_bwd(lib, s) == code
    assert lib.falcon_selective_scan_bwd_workspace_bytes(s) == 0


def test_scan_refuses_bad_pointers(lib):
    s = _scan_shape()
    assert _scan_fwd(lib, None) == -1
    assert _scan_fwd(lib, s, u=None) == -1
    assert _scan_fwd(lib, s, A=None) == -1
    assert _scan_fwd(lib, s, h=None) == -1
    assert _scan_fwd(lib, s, z=_p()) == -1  # a gate without its strides
    assert _scan_fwd(lib, s, y=_p(0x10002)) == -4
    assert _scan_fwd(lib, s, h=_p(0x10001)) == -4
    assert _scan_fwd(lib, s, us=_strides(batch=-4)) == -8
    assert _scan_fwd(lib, s, bs=_strides(head=-4)) == -8
    assert _scan_fwd(lib, _scan_shape(B=0), u=None, A=None) == 0
    assert _scan_bwd(lib, s, dy=None) == -1
    assert _scan_bwd(lib, s, dA=None) == -1
    assert _scan_bwd(lib, s, z=_p()) == -1  # a gate without room for its gradient
    assert _scan_bwd(lib, s, dz=_p()) == -8
    assert _scan_bwd(lib, s, ws=None) == -5
    assert _scan_bwd(lib, s, have=256) == -5
    assert _scan_bwd(lib, s, ws=_p(0x10010)) == -4


def test_scan_step_refuses(lib):
    def step(N=2, D=16, G=2, S=16, dt=F32, u=_p(), us=16, A=_p(), h=_p(), pool=2, y=_p()):
        st = _strides()
        return lib.falcon_selective_scan_step(N, D, G, S, dt, 1, u, us, _p(), 16, A, _p(), st,
                                              _p(), st, None, None, 0, None, h, pool, None, None,
                                              y, None)
    assert step(N=-1) == -2
    assert step(S=0) == -2
    assert step(S=200) == -2
    assert step(G=5) == -2
    assert step(pool=-1) == -2
    assert step(dt=4) == -3
    assert step(us=-1) == -8
    assert step(u=None) == -1
    assert step(h=None) == -1
    assert step(h=_p(0x10002)) == -4
    assert step(N=0, u=None) == 0


def test_clip_refuses(lib):
    from delta_rule_attention_gb300.block import falcon_grad

    def clip(grad=0x10000, out=0x10000, count=8, dtype=F32, n=1, max_norm=1.0, eps=1e-6,
             norm=_p(), ws=_p(), have=1 << 30, table=True):
        t = (falcon_grad * 1)()
        t[0].grad, t[0].out, t[0].count, t[0].dtype = grad, out, count, dtype
        return lib.falcon_clip_grad_norm(t if table else None, n, max_norm, eps, norm, ws, have,
                                         None)
    assert clip(n=-1) == -2
    assert clip(count=-1) == -2
    assert clip(dtype=2) == -3
    assert clip(table=False) == -1
    assert clip(norm=None) == -1
    assert clip(grad=None) == -1
    assert clip(out=None) == -1
    assert clip(grad=0x10002) == -4
    assert clip(grad=0x10001, dtype=BF16) == -4
    assert clip(max_norm=-1.0) == -8
    assert clip(max_norm=float("nan")) == -8
    assert clip(eps=-1.0) == -8
    assert clip(ws=None) == -5
    assert clip(have=8) == -5
    assert clip(ws=_p(0x10008)) == -4


def test_binding_refuses_host_tensors_and_wrong_types():
    import delta_rule_attention_gb300 as falcon
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        falcon.falcon_short_conv_fwd(x, w)  # not on a GPU
    with pytest.raises(TypeError):
        falcon.falcon_short_conv_fwd(x.half(), w)
    with pytest.raises(ValueError):
        falcon.falcon_short_conv_fwd(x[0], w)
    with pytest.raises(ValueError):
        falcon.falcon_short_conv_fwd(x, w, activation="relu")
    with pytest.raises(TypeError):
        falcon.falcon_clip_grad_norm([torch.zeros(3).double()], 1.0)
    with pytest.raises(ValueError):
        falcon.falcon_clip_grad_norm([], 1.0)
