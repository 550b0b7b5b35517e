"""Results of the convolution and the scan that lie on one another, or on what other
threads still read: refused, with nothing launched (no GPU needed)."""
import ctypes
import os
import shutil

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")

F32, BAD_ARG = 1, -8


@pytest.fixture(scope="module")
def lib():
    from delta_rule_attention_gb300 import _build
    _build.build()
    import delta_rule_attention_gb300 as falcon
    return falcon.load_library()


def _p(addr):
    return ctypes.c_void_p(addr)


def _conv(lib, x=0x10000, y=0x20000, dy=0x30000, dx=0x40000, back=False, ys=(1024, 0, 16), **kw):
    from delta_rule_attention_gb300.block import falcon_conv_shape, falcon_strides
    base = dict(B=2, H=1, T=8, m=16, width=4, dtype=F32, activation=1)
    base.update(kw)
    s = falcon_conv_shape(*[base[f] for f, _ in falcon_conv_shape._fields_])
    st, out = falcon_strides(1024, 512, 16), falcon_strides(*ys)
    if not back:
        return lib.falcon_short_conv_fwd(s, _p(x), st, _p(0x50000), None, None, None, _p(y), out,
                                         None, None)
    return lib.falcon_short_conv_bwd(s, _p(x), st, _p(0x50000), None, None, None, _p(dy), st, None,
                                     _p(dx), out, _p(0x60000), None, None, _p(0x70000), 1 << 40,
                                     None)


def test_conv_refuses_to_write_where_it_reads(lib):
    """A run of tokens reads the rows before it, which another thread would overwrite."""
    assert _conv(lib, y=0x10000) == BAD_ARG
    assert _conv(lib, back=True, dx=0x10000) == BAD_ARG
    assert _conv(lib, back=True, dx=0x30000) == BAD_ARG


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("ys,kw", [((1024, 0, 0), {}), ((0, 0, 16), {}), ((1024, 0, 16), dict(H=2))])
def test_conv_refuses_results_that_lie_on_one_another(lib, back, ys, kw):
    assert _conv(lib, back=back, ys=ys, **kw) == BAD_ARG


@pytest.mark.parametrize("ys", [(1024, 0, 0), (0, 0, 16)])
def test_scan_refuses_results_that_lie_on_one_another(lib, ys):
    from delta_rule_attention_gb300.block import falcon_scan_shape, falcon_strides
    s, st = falcon_scan_shape(2, 8, 16, 1, 16, F32, 1), falcon_strides(1024, 0, 16)
    assert lib.falcon_selective_scan_fwd(
        s, _p(0x10000), st, _p(0x20000), st, _p(0x30000), _p(0x40000), st, _p(0x50000), st, None,
        None, None, None, None, None, _p(0x60000), falcon_strides(*ys), _p(0x70000), None) == BAD_ARG


def test_scan_gradient_refuses_to_write_the_states_it_reads(lib):
    """dh0 over h0: the walk over the chunks reads one in one block and writes the other in
    another.  Over dh_T it may lie (the workspace is too small here, so that nothing runs)."""
    from delta_rule_attention_gb300.block import falcon_scan_shape, falcon_strides
    s, st = falcon_scan_shape(2, 8, 16, 1, 16, F32, 1), falcon_strides(1024, 0, 16)

    def call(h0, dh_T, dh0):
        p = [_p(0x100000 + 0x10000 * i) for i in range(12)]
        return lib.falcon_selective_scan_bwd(
            s, p[0], st, p[1], st, p[2], p[3], st, p[4], st, None, None, None, None, h0, None, p[5],
            st, dh_T, p[6], p[7], p[8], p[9], p[10], None, None, None, dh0, p[11], 256, None)

    a, b = _p(0x800000), _p(0x900000)
    assert call(a, b, a) == BAD_ARG
    assert call(a, b, b) == -5
