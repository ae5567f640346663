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


FORM_OF = r"""
#include <stdio.h>
#include <string.h>
#include <map>
#include <string>
#include "moe_plan.hpp"
using namespace fgb;
static std::string form(int T, int E, int k, int H, int I) {
  const bool late = use_late(T, k, E, H, I);
  const int want = late ? 1 : gate_up_slices(T, k, E, H, I), per = (H / 128 + want - 1) / want;
  const int slices = (H / 128 + per - 1) / per;
  char b[96];
  snprintf(b, sizeof b, "%s tiles%d %s %s %s", late ? "late" : fused_prep(T, H) ? "fused" : "prep",
           T <= 16 ? 1 : T <= 32 ? 2 : 4, slices > 1 ? "gate_up_sliced" : "gate_up_whole",
           down_wide(H) ? "down_wide" : "down_narrow", down_slices(T, k, E, H, I) > 1 ? "down_sliced" : "down_whole");
  return b;
}
int main(int argc, char** argv) {
  int T, E, k, H, I;
  while (scanf("%d %d %d %d %d", &T, &E, &k, &H, &I) == 5) printf("shape %s\n", form(T, E, k, H, I).c_str());
  if (argc < 2 && getchar() != EOF) return 1;
  // every form that some call takes, with the first such call
  std::map<std::string, std::string> seen;
  const int Es[] = {1, 2, 4, 8, 16, 32, 64, 128, 256, 512, 1024}, ks[] = {1, 2, 4, 8, 16};
  for (int T = 1; T <= 64; ++T)
    for (int E : Es)
      for (int k : ks)
        if (k <= E)
          for (int h = 1; h <= 256; h += h < 16 ? 1 : 9)
            for (int i = 1; i <= 256; i += i < 16 ? 1 : 9) {
              char b[64];
              snprintf(b, sizeof b, "%dx%dx%dx%dx%d", T, E, k, 128 * h, 128 * i);
              seen.emplace(form(T, E, k, 128 * h, 128 * i), b);
            }
  for (auto& f : seen) printf("form %s %s\n", f.first.c_str(), f.second.c_str());
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


def test_every_launch_form_has_a_test_shape(tmp_path):
    """Every form that the rules choose (quantization late, in gate+up or by the prep launch; one to four row
    tiles; gate+up and down whole or sliced; down's width) is met by a shape of the GPU tests."""
    from tests.test_gpu_moe_ffn import SHAPES
    from tests.test_gpu_moe_forms import SHAPES as MORE

    text = "".join("%d %d %d %d %d\n" % s for s in SHAPES + MORE)
    rows = compile_and_run(tmp_path, FORM_OF, text)
    tested = {tuple(r[1:]) for r in rows if r[0] == "shape"}
    forms = {tuple(r[1:-1]): r[-1] for r in rows if r[0] == "form"}
    assert len(forms) >= 12
    missing = {f: at for f, at in forms.items() if f not in tested}
    assert not missing, missing
