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


@pytest.mark.parametrize("T", [1, 2, 7, 128, 77824, 2 ** 30 + 1, 2 ** 31 - 1])
def test_rows_further_on(tmp_path, T):
    """A block's way through the rows of a norm, to the end of the problem and a few rows
    behind it, against division in 64 bits: rows of up to 2^31 - 1 tokens."""
    B = (2 ** 31 - 1) // T
    run_on_host(tmp_path, f"""
  const long long T = {T}LL, B = {B}LL;
  for (long long step : {{1LL, 2LL, 19456LL, 38912LL, 77824LL}})
    for (long long row : {{0LL, 1LL, step - 1, T / 2, T - 2 * step, T - step, T - 1,
                           B * T - 3 * step, B * T - step, B * T - 1}}) {{
      if (row < 0) continue;
      unsigned b = (unsigned)(row / T);
      int t = (int)(row % T);
      for (int i = 0; i < 8 && row < B * T; ++i) {{
        row += step;
        falcon::advance_row(b, t, (int)(step / T), (int)(step % T), (int)T);
        if (b != row / T || t != row % T) {{
          printf("step %lld row %lld: (%u, %d)\\n", step, row, b, t);
          return 1;
        }}
      }}
    }}
  return 0;""", "gated_norm.cuh")
