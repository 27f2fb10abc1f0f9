"""Arithmetic of the serving kernels that the host shares with them, compiled and run on the host (no GPU needed)."""
import subprocess

from gated_delta_rule_linear_gb300 import build as labuild

RUNS = r"""
#include <climits>
#include <cstdio>
#include "la_serve_internal.h"

int main() {
  const int totals[] = {0, 1, 151, 152, 153, 100000, INT_MAX / 2 + 1, 2147418176, INT_MAX - 1, INT_MAX};
  const unsigned grids[] = {1, 2, 152, 304, 608};
  int bad = 0;
  for (int total : totals)
    for (unsigned ctas : grids) {
      const int share = la::share_of(total, ctas);
      int at = 0;
      for (unsigned c = 0; c < ctas; ++c) {
        const la::UnitRun r = la::run_of(c, share, total);
        if (r.first != at || r.end < r.first || r.end > total) {
          if (bad++ < 5) printf("%d units, CTA %u of %u: %d..%d behind %d\n", total, c, ctas, r.first, r.end, at);
        }
        at = r.end;
      }
      if (at != total && bad++ < 5) printf("%d units over %u CTAs: %d\n", total, ctas, at);
    }
  return bad != 0;
}
"""


def test_runs_of_units_are_all_of_them(tmp_path):
    """Every unit is one CTA's, in order, up to the largest number of units that an int holds."""
    src, exe = tmp_path / "runs.cu", tmp_path / "runs"
    src.write_text(RUNS)
    subprocess.run([labuild.nvcc_path(), *labuild.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", labuild.INCLUDE, "-I",
                    labuild.CSRC, str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
