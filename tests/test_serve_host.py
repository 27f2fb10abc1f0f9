"""What the host decides for the serving kernels, and the arithmetic that it shares with them (no GPU needed)."""
import subprocess

import pytest

import gated_delta_rule_linear_gb300 as la
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


A = 0x10000  # fake, aligned device addresses: never dereferenced by a refused call


@pytest.mark.parametrize("n,H,Hk,d,f32,pages", [
    (65, 1, 1, 64, 0, 2047), (33, 2, 2, 128, 0, 2047), (13, 80, 1, 256, 0, 2 ** 31 - 1),
    (33, 1, 1, 128, 1, 2047), (33, 4, 1, 256, 1, 2047), (17, 8, 1, 256, 1, 2047), (9, 16, 1, 256, 1, 2 ** 31 - 1),
])
def test_attention_of_tables_that_are_too_large(n, H, Hk, d, f32, pages):
    """Refused as an argument, before there is a device: twice what the header allows, as (2^31 - 2^16) / 2^20 pages of 2^20
    places or more are counted for each part."""
    labuild.build()
    page = 1 << 20
    rc = la.la_paged_attn(A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A, 7 * A, n, H, Hk, d, page, 9, pages, pages, 0, 0, 0.125, H * d,
                          page * Hk * d, la.LA_F32 if f32 else 0, None)
    assert rc == la.CONSTANTS["LA_ERR_INVALID_ARG"], rc
    assert "too large" in la.la_last_error()
