"""The scan gradient's workspace stays in proportion to its tensors at every state size
(no GPU needed)."""
import os
import shutil

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc to build the library")


@pytest.fixture(scope="module")
def lib():
    from delta_rule_attention_gb300 import _build
    _build.build()
    import delta_rule_attention_gb300 as falcon
    return falcon.load_library()


@pytest.mark.parametrize("N", [4, 16, 17, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("B,T,D,G", [(8, 2048, 2048, 1), (8, 4096, 4096, 1), (8, 2048, 2048, 8),
                                     (1, 65536, 2048, 1), (32, 2048, 64, 1)])
def test_scan_gradient_workspace(lib, B, T, D, G, N):
    """A state and an adjoint for every 32 tokens, padded to a power of two; parameter sums
    of at most a quarter of that; dB and dC terms of 2 GB, or of one fp32 copy of
    dB and dC where that is larger, and their sum; a step sum."""
    from delta_rule_attention_gb300.block import falcon_scan_shape
    need = lib.falcon_selective_scan_bwd_workspace_bytes(falcon_scan_shape(B, T, D, G, N, 0, 1))
    padded = 4
    while padded < N:
        padded *= 2
    chunks = (T + 31) // 32
    states = 2 * 4 * B * chunks * D * padded
    terms = 2 * 4 * B * T * G * padded
    sums = states // 2 + 4 * B * D * (3 * chunks + padded) + 4096
    assert need <= states + sums + max(2 << 30, terms) + terms
