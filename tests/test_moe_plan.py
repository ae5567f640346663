"""CPU: the mixture-of-experts layer's plan (csrc/moe_plan.hpp), compiled with g++ into a small program that
prints what it is asked for."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fine_grained_block_amd", "csrc")

LDS_OF = r"""
#include <stdio.h>
#include "moe_plan.hpp"
using namespace fgb;
int main() {  // every segment length and token count: codes and scales of each wave, bytes in all
  for (int seg = 1; seg <= 64; ++seg)
    for (int T = 1; T <= kTile; ++T) {
      if (seg * T > kLateBlocks) continue;
      printf("%d %d %d", seg, T, late_bytes(seg, T));
      for (int w = 0; w < kDownWaves; ++w) printf(" %d %d", late_codes_at(w, seg, T), late_scales_at(w, seg, T));
      printf("\n");
    }
}
"""


def compile_and_run(tmp_path, source, text=""):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    src, exe = tmp_path / "plan.cpp", str(tmp_path / "plan")
    src.write_text(source)
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", exe], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
    assert r.returncode == 0
    return [line.split() for line in r.stdout.splitlines()]


def test_late_quantization_lds(tmp_path):
    """Late quantization's LDS: 16-byte accesses to the codes are aligned, scales too, the waves' areas are
    apart and inside the launch's bytes (which begin on a 16-byte boundary: whole columns of sums)."""
    rows = [[int(v) for v in r] for r in compile_and_run(tmp_path, LDS_OF)]
    assert len(rows) > 150
    for seg, T, total, *at in rows:
        areas = []
        for codes, scales in zip(at[::2], at[1::2]):
            assert codes % 16 == 0 and scales % 4 == 0, (seg, T)
            areas += [(codes, codes + seg * T * 128), (scales, scales + seg * T * 4)]
        areas.sort()
        assert areas[0][0] >= 0 and areas[-1][1] <= total
        assert all(a[1] <= b[0] for a, b in zip(areas, areas[1:])), (seg, T)
        # beside 32 KB of weight tiles and the waves' sums of up to 32 columns
        assert 8 * 2 * 2048 + 8 * T * 32 * 4 + total <= 160 << 10
