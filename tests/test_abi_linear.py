"""Argument checks of the linear attention block's entry points: refused before a device
is touched, with nothing launched (no GPU needed)."""
import ctypes
import os
import shutil

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")

BF16, F32 = 0, 1
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ARG = -1, -2, -3, -4, -5, -8


@pytest.fixture(scope="module")
def lib():
    from delta_rule_attention_gb300 import _build
    _build.build()
    import delta_rule_attention_gb300 as falcon
    return falcon.load_library()


def p(addr):
    return ctypes.c_void_p(addr)


# one address a tensor: none lies on another
AT = {n: p(0x100000 * (i + 1)) for i, n in enumerate(
    "q k v log_decay S0 lengths o S_out ws dO dS_T dq dk dv dS0 h weight z scale x next_weight "
    "out next dout dnext dx dh dz dweight dscale dnext_weight S slots fresh".split())}


def strides(batch=4096, head=1024, time=16):
    from delta_rule_attention_gb300.block import falcon_strides
    return falcon_strides(batch, head, time)


def decay_shape(**kw):
    from delta_rule_attention_gb300.linear import falcon_decay_shape
    base = dict(B=2, H=2, T=8, m=16, dv=16, dtype=F32, scale=0.25)
    base.update(kw)
    return falcon_decay_shape(*[base[f] for f, _ in falcon_decay_shape._fields_])


def norm_shape(**kw):
    from delta_rule_attention_gb300.linear import falcon_norm_shape
    base = dict(B=2, H=2, T=8, m=16, dtype=F32, gate=1, eps=1e-6)
    base.update(kw)
    return falcon_norm_shape(*[base[f] for f, _ in falcon_norm_shape._fields_])


def a(kw, name):
    return kw.get(name, AT[name])


def s(kw, name):
    return kw.get(name + "_s", strides())


def fwd(lib, shape, have=1 << 40, **kw):
    act = lambda n: (a(kw, n), s(kw, n))  # noqa: E731
    return lib.falcon_decay_attn_fwd(shape, *act("q"), *act("k"), *act("v"), a(kw, "log_decay"),
                                     a(kw, "S0"), a(kw, "lengths"), *act("o"), a(kw, "S_out"),
                                     a(kw, "ws"), have, None)


def bwd(lib, shape, have=1 << 40, **kw):
    act = lambda n: (a(kw, n), s(kw, n))  # noqa: E731
    return lib.falcon_decay_attn_bwd(
        shape, *act("q"), *act("k"), *act("v"), a(kw, "log_decay"), a(kw, "S0"), a(kw, "lengths"),
        *act("dO"), a(kw, "dS_T"), *act("dq"), *act("dk"), *act("dv"), a(kw, "dS0"), a(kw, "ws"),
        have, None)


def step(lib, shape, pool=4, **kw):
    act = lambda n: (a(kw, n), s(kw, n))  # noqa: E731
    return lib.falcon_decay_attn_step(shape, *act("q"), *act("k"), *act("v"), a(kw, "log_decay"),
                                      a(kw, "S"), pool, a(kw, "slots"), a(kw, "fresh"),
                                      a(kw, "o"), None)


BAD_DECAY = [(dict(B=-1), SHAPE), (dict(H=-1), SHAPE), (dict(T=-1), SHAPE), (dict(m=0), SHAPE),
             (dict(m=129), SHAPE), (dict(dv=0), SHAPE), (dict(dv=129), SHAPE),
             (dict(B=1 << 40), SHAPE), (dict(B=1 << 20, H=1 << 20), SHAPE),
             (dict(T=1 << 40), SHAPE), (dict(dtype=2), DTYPE),
             (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG)]


@pytest.mark.parametrize("bad,code", BAD_DECAY)
def test_decay_refuses_bad_shapes(lib, bad, code):
    assert fwd(lib, decay_shape(**bad)) == code
    assert bwd(lib, decay_shape(**bad)) == code
    if "T" not in bad:
        assert step(lib, decay_shape(**bad)) == code
    assert lib.falcon_decay_attn_workspace_bytes(decay_shape(**bad)) == 0
    assert lib.falcon_decay_attn_bwd_workspace_bytes(decay_shape(**bad)) == 0


def test_decay_forward_refuses(lib):
    sh = decay_shape()
    assert fwd(lib, None) == NULL
    for name in ("q", "k", "v", "o", "log_decay", "q_s", "k_s", "v_s", "o_s"):
        assert fwd(lib, sh, **{name: None}) == NULL, name
    for name in ("q", "k", "v", "o", "log_decay", "S0", "lengths", "S_out"):
        assert fwd(lib, sh, **{name: p(0x9000002)}) == ALIGN, name
    assert fwd(lib, decay_shape(dtype=BF16), q=p(0x9000001)) == ALIGN
    for name in ("q", "k", "v", "o"):
        assert fwd(lib, sh, **{name + "_s": strides(time=-16)}) == ARG, name
    assert fwd(lib, sh, o_s=strides(head=0)) == ARG
    assert fwd(lib, sh, o_s=strides(time=0)) == ARG
    for name in ("q", "k", "v", "S0", "S_out", "log_decay"):
        assert fwd(lib, sh, o=AT[name]) == ARG, name
    for name in ("q", "k", "v", "log_decay"):
        assert fwd(lib, sh, S_out=AT[name]) == ARG, name
    assert lib.falcon_decay_attn_workspace_bytes(sh) > 0
    assert fwd(lib, sh, ws=None) == WORKSPACE
    assert fwd(lib, sh, have=4) == WORKSPACE
    assert fwd(lib, sh, ws=p(0x9000010)) == ALIGN
    assert fwd(lib, decay_shape(B=0), q=None, o=None, ws=None) == 0


def test_decay_backward_refuses(lib):
    sh = decay_shape()
    for name in ("q", "k", "v", "dO", "dq", "dk", "dv", "log_decay", "dO_s", "dq_s", "dk_s",
                 "dv_s"):
        assert bwd(lib, sh, **{name: None}) == NULL, name
    for name in ("dO", "dq", "dk", "dv", "dS_T", "dS0"):
        assert bwd(lib, sh, **{name: p(0x9000002)}) == ALIGN, name
    for name in ("dq", "dk", "dv"):
        assert bwd(lib, sh, **{name + "_s": strides(batch=-1)}) == ARG
        assert bwd(lib, sh, **{name + "_s": strides(batch=0)}) == ARG
        for other in ("q", "k", "v", "dO", "S0", "dS_T", "dS0"):
            assert bwd(lib, sh, **{name: AT[other]}) == ARG, (name, other)
    assert bwd(lib, sh, dq=AT["dk"]) == ARG and bwd(lib, sh, dv=AT["dk"]) == ARG
    assert bwd(lib, sh, dS0=AT["S0"]) == ARG
    assert bwd(lib, sh, ws=None) == WORKSPACE
    assert bwd(lib, sh, have=4) == WORKSPACE
    assert bwd(lib, decay_shape(H=0), q=None, ws=None) == 0


def test_decay_step_refuses(lib):
    sh = decay_shape()
    for name in ("q", "k", "v", "S", "o", "log_decay", "q_s", "k_s", "v_s"):
        assert step(lib, sh, **{name: None}) == NULL, name
    for name in ("q", "k", "v", "S", "o", "slots"):
        assert step(lib, sh, **{name: p(0x9000002)}) == ALIGN, name
    assert step(lib, sh, pool=-1) == SHAPE
    assert step(lib, sh, pool=1, slots=None) == SHAPE
    assert step(lib, sh, q_s=strides(head=-1)) == ARG
    assert step(lib, sh, o=AT["v"]) == ARG
    assert step(lib, decay_shape(B=0), q=None, S=None) == 0


def nfwd(lib, shape, **kw):
    act = lambda n: (a(kw, n), s(kw, n))  # noqa: E731
    return lib.falcon_gated_norm_fwd(shape, *act("h"), a(kw, "weight"), *act("z"), a(kw, "scale"),
                                     *act("x"), a(kw, "next_weight"), a(kw, "lengths"),
                                     *act("out"), *act("next"), None)


def nbwd(lib, shape, have=1 << 40, **kw):
    act = lambda n: (a(kw, n), s(kw, n))  # noqa: E731
    return lib.falcon_gated_norm_bwd(
        shape, *act("h"), a(kw, "weight"), *act("z"), a(kw, "scale"), *act("out"),
        a(kw, "next_weight"), a(kw, "lengths"), *act("dout"), *act("dnext"), *act("dx"),
        *act("dh"), *act("dz"), a(kw, "dweight"), a(kw, "dscale"), a(kw, "dnext_weight"),
        a(kw, "ws"), have, None)


BAD_NORM = [(dict(B=-1), SHAPE), (dict(H=0), SHAPE), (dict(T=-1), SHAPE), (dict(m=0), SHAPE),
            (dict(H=2, m=4097), SHAPE), (dict(H=8193, m=1), SHAPE), (dict(B=1 << 20, T=1 << 20),
                                                                     SHAPE),
            (dict(dtype=7), DTYPE), (dict(gate=3), ARG), (dict(gate=-1), ARG),
            (dict(eps=0.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=-1.0), ARG)]


@pytest.mark.parametrize("bad,code", BAD_NORM)
def test_norm_refuses_bad_shapes(lib, bad, code):
    assert nfwd(lib, norm_shape(**bad)) == code
    assert nbwd(lib, norm_shape(**bad)) == code
    assert lib.falcon_gated_norm_bwd_workspace_bytes(norm_shape(**bad)) == 0


def test_norm_forward_refuses(lib):
    sh = norm_shape()
    assert nfwd(lib, None) == NULL
    for name in ("out", "out_s", "h_s", "z_s", "x_s", "next", "next_s", "next_weight"):
        assert nfwd(lib, sh, **{name: None}) == NULL, name
    for name in ("h", "z", "x", "out", "next", "weight", "scale", "next_weight", "lengths"):
        assert nfwd(lib, sh, **{name: p(0x9000002)}) == ALIGN, name
    for name in ("h", "z", "x", "out", "next"):
        assert nfwd(lib, sh, **{name + "_s": strides(batch=-1)}) == ARG, name
    for name in ("h", "z", "weight", "scale", "next_weight"):
        assert nfwd(lib, sh, out=AT[name]) == ARG, name
        assert nfwd(lib, sh, next=AT[name]) == ARG, name
    assert nfwd(lib, sh, next=AT["x"]) == ARG and nfwd(lib, sh, next=AT["out"]) == ARG
    assert nfwd(lib, sh, out=AT["x"], out_s=strides(time=32)) == ARG
    assert nfwd(lib, sh, out_s=strides(time=0)) == ARG
    # without h there are x and the next norm only
    assert nfwd(lib, sh, h=None) == ARG
    bare = dict(h=None, out=None, weight=None, scale=None, z=None)
    assert nfwd(lib, sh, **bare, x=None) == NULL
    assert nfwd(lib, sh, **bare, next=None) == NULL
    assert nfwd(lib, norm_shape(B=0), h=p(0x10)) == 0


def test_norm_backward_refuses(lib):
    sh = norm_shape()
    for name in ("dh", "dh_s", "dz", "dz_s", "out", "dnext", "dout_s", "dx_s"):
        assert nbwd(lib, sh, **{name: None}) == NULL, name
    assert nbwd(lib, sh, z=None) == NULL  # dz without z
    assert nbwd(lib, sh, next_weight=None, dnext_weight=None) == NULL  # dnext without it
    assert nbwd(lib, sh, next_weight=None, dnext=None, dout=None, dnext_weight=None) == NULL
    assert nbwd(lib, sh, scale=None) == ARG  # dscale without scale
    assert nbwd(lib, sh, next_weight=None, dnext=None) == ARG
    assert nbwd(lib, sh, h=None) == ARG
    for name in ("dout", "dnext", "dx", "dh", "dz", "dweight", "dscale", "dnext_weight"):
        assert nbwd(lib, sh, **{name: p(0x9000002)}) == ALIGN, name
    for name in ("dx", "dh", "dz"):
        assert nbwd(lib, sh, **{name + "_s": strides(batch=0)}) == ARG, name
        for other in ("h", "z", "out", "dnext", "weight"):
            assert nbwd(lib, sh, **{name: AT[other]}) == ARG, (name, other)
    assert nbwd(lib, sh, dh=AT["dout"]) == ARG and nbwd(lib, sh, dz=AT["dout"]) == ARG
    assert nbwd(lib, sh, dx=AT["dh"]) == ARG and nbwd(lib, sh, dz=AT["dx"]) == ARG
    assert nbwd(lib, sh, dx=AT["dout"], dx_s=strides(time=32)) == ARG
    assert nbwd(lib, sh, dweight=AT["weight"]) == ARG and nbwd(lib, sh, dscale=AT["dweight"]) == ARG
    assert lib.falcon_gated_norm_bwd_workspace_bytes(sh) > 0
    assert nbwd(lib, sh, ws=None) == WORKSPACE
    assert nbwd(lib, sh, have=4) == WORKSPACE
    assert nbwd(lib, sh, ws=p(0x9000008)) == ALIGN
