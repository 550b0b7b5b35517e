"""Index arithmetic of the linear attention block's kernels, compiled for the host and
compared with plain loops (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from delta_rule_attention_gb300 import _build

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and
                                not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="needs nvcc")


def run_on_host(tmp_path, body, *headers):
    """Compiles a program around `body`, which returns 0, and runs it."""
    src, exe = tmp_path / "host.cu", tmp_path / "host"
    src.write_text("".join(f'#include "{h}"\n' for h in headers) +
                   "#include <cstdio>\nint main() {\n" + body + "\n}\n")
    subprocess.run([_build._nvcc(), *_build.ARCH, "-std=c++17", "-I" + _build.INCLUDE,
                    "-I" + _build.CSRC, "-cudart", "static", "-o", str(exe), str(src)], check=True,
                   capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_last_phase_of_a_ring(tmp_path):
    """What a block waits for at its end: the phase that the last use of each barrier
    completed, found by going through the uses."""
    run_on_host(tmp_path, """
  for (int stages = 1; stages <= 4; ++stages)
    for (int n = 0; n < 40; ++n) {
      int phases[4] = {0, 0, 0, 0};
      for (int c = 0; c < n; ++c) ++phases[c % stages];
      for (int s = 0; s < stages && s < n; ++s)
        if (falcon::last_phase(n, stages, s) != phases[s] - 1) {
          printf("n %d stages %d barrier %d\\n", n, stages, s);
          return 1;
        }
      for (int s = n; s < stages; ++s)
        if (phases[s]) return 2;
    }
  return 0;""", "linear_tc.cuh")
