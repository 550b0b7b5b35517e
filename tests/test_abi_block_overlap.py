"""Clipping into memory that two blocks would write, or that one writes while another
reads it: refused, with nothing launched (no GPU needed)."""
import ctypes
import os
import shutil

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")

BF16, F32 = 0, 1
BAD_ARG, WORKSPACE = -8, -5


@pytest.fixture(scope="module")
def lib():
    from delta_rule_attention_gb300 import _build
    _build.build()
    import delta_rule_attention_gb300 as falcon
    return falcon.load_library()


def _p(addr):
    return ctypes.c_void_p(addr)


def _clip(lib, rows):
    """rows of (grad, out, count, dtype); the workspace is too small, so that a set that
    is not refused for its addresses is refused for that."""
    from delta_rule_attention_gb300.block import falcon_grad
    t = (falcon_grad * len(rows))()
    for i, (grad, out, count, dtype) in enumerate(rows):
        t[i].grad, t[i].out, t[i].count, t[i].dtype = grad, out, count, dtype
    return lib.falcon_clip_grad_norm(t, len(rows), 1.0, 1e-6, _p(0x900000), _p(0xa00000), 8, None)


def _placed(*rows):
    return [(a, a, n, F32) for a, n in rows]


@pytest.mark.parametrize("rows", [
    _placed((0x10000, 8), (0x10000, 8)),                   # a gradient named twice
    _placed((0x10000, 8), (0x20000, 8), (0x10000, 8)),
    _placed((0x20000, 8), (0x10000, 8), (0x20000, 8)),
    _placed((0x10000, 8), (0x1001c, 8)),                   # one element shared
    _placed((0x1001c, 8), (0x10000, 8)),
    _placed((0x10000, 100), (0x10040, 1), (0x20000, 4)),   # one inside another
    [(0x10000, 0x10000, 8, F32), (0x1001e, 0x1001e, 1, BF16)],
    [(0x10000, 0x30000, 8, F32), (0x20000, 0x30000, 8, F32)],   # two results in one place
    [(0x10000, 0x20000, 8, F32), (0x20000, 0x30000, 8, F32)],   # a result on another's input
    [(0x20000, 0x30000, 8, F32), (0x10000, 0x20010, 8, F32)],
    [(0x10000, 0x10004, 8, F32)],                               # on its own, moved
], ids=range(11))
def test_clip_refuses_results_that_overlap(lib, rows):
    assert _clip(lib, rows) == BAD_ARG


@pytest.mark.parametrize("rows", [
    _placed((0x10000, 8), (0x10020, 8), (0x10040, 1)),     # packed one behind the other
    _placed((0x10040, 1), (0x10020, 8), (0x10000, 8)),
    _placed((0x10000, 8), (0x10000, 0), (0x20000, 8)),     # nothing at an address
    _placed((0x10010, 0), (0x10000, 8)),
    [(0x10000, 0x30000, 8, F32), (0x10000, 0x40000, 8, F32)],   # one input, two results
    [(0x10000, 0x10020, 8, F32), (0x10040, 0x10060, 8, F32)],   # interleaved
    [(0x10040, 0x10060, 8, F32), (0x10000, 0x10020, 8, F32), (0x10080, 0x10080, 4, F32)],
], ids=range(7))
def test_clip_takes_results_that_do_not(lib, rows):
    assert _clip(lib, rows) == WORKSPACE


def test_clip_of_many_unordered_tensors(lib):
    places = [0x100000 + 64 * (i * 7919 % 5000) for i in range(5000)]
    assert _clip(lib, _placed(*((a, 16) for a in places))) == WORKSPACE
    assert _clip(lib, _placed(*((a, 16) for a in places), (places[4321] + 60, 1))) == BAD_ARG
