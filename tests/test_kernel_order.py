"""The order in which kernels take tensor memory and let the launch behind them start, read from
their sources (no GPU needed).

A block of the launch behind allocates tensor memory and holds it while it waits for this
grid to complete.  If it came first, this grid's block would wait for that memory, and
neither would go on."""
import glob
import os
import re

import pytest

from delta_rule_attention_gb300 import _build

TRIGGER, ALLOC = "griddepcontrol.launch_dependents", "tmem_alloc("


def kernels():
    """(file, name, body) of every kernel that does both."""
    for path in sorted(glob.glob(os.path.join(_build.CSRC, "*.cu"))):
        src = open(path).read()
        src = re.sub(r"//[^\n]*", "", src)
        for m in re.finditer(r"__global__", src):
            # the body opens at the first line that ends in a brace
            start = src.index("{\n", m.end())
            depth, at = 0, start
            while True:
                depth += {"{": 1, "}": -1}.get(src[at], 0)
                if depth == 0:
                    break
                at += 1
            body = src[start:at]
            if TRIGGER in body and ALLOC in body:
                name = re.findall(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\([^;]*?\)\s*\n?", "",
                                                       src[m.end():start], count=1))
                yield os.path.basename(path), (name or ["kernel"])[0], body


CASES = list(kernels())


def test_the_kernels_are_found():
    assert len(CASES) >= 6 and {c[0] for c in CASES} >= {
        "chunk_tc.cu", "decay_attn_tc.cu", "falcon2_tc.cu", "falcon2a_tc.cu", "falcon3a_tc.cu"}


@pytest.mark.parametrize("case", range(len(CASES)), ids=[f"{f}-{n}-{i}" for i, (f, n, _) in
                                                         enumerate(CASES)])
def test_tensor_memory_comes_before_the_launch_behind(case):
    _, _, body = CASES[case]
    alloc, trigger = body.index(ALLOC), body.index(TRIGGER)
    assert alloc < trigger
    # and every warp knows of it: the first one that lets the launch behind start does so for
    # the block
    assert "__syncthreads()" in body[alloc:trigger]
