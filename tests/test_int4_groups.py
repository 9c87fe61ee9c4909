"""The scale groups that a phase of the streamed int4 product touches, to the
largest K and group that nvfp4_int4_gemm accepts (host arithmetic, no GPU): the
header's function compiled with overflow traps, against 64-bit arithmetic."""

import os
import subprocess

from conftest import ROOT

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "int4_groups.hpp"

int main() {
  const int64_t top = (int64_t)1 << 30;
  const int64_t sizes[] = {32, 64, 96, 160, 256, 2080, 4096, 8224, 151936, (int64_t)1 << 22, top - 4096, top - 128, top};
  const int64_t spans[] = {256, 512, 2816, 4096};
  long checked = 0;
  for (int64_t K : sizes)
    for (int64_t group : {(int64_t)32, (int64_t)64, (int64_t)128, (int64_t)384, (int64_t)1 << 20, K / 2, K}) {
      if (group < 32 || K % group) continue;
      for (int64_t span : spans) {
        const int64_t phases = (K + span - 1) / span;
        // the first and the last phases of long rows
        for (int64_t ph = 0; ph < phases; ph = ph == 64 && phases > 200 ? phases - 64 : ph + 1) {
          const int64_t k0 = ph * span, k1 = k0 + span < K ? k0 + span : K;
          const int64_t first = k0 / group, count = (k1 + group - 1) / group - first;
          const nvfp4::I4Groups g = nvfp4::i4_groups((int)k0, (int)span, (int)K, (int)group);
          if (g.first != first || g.count != count || count < 1) {
            std::printf("K %ld group %ld span %ld phase %ld: %d + %d, not %ld + %ld\n", (long)K, (long)group, (long)span,
                        (long)ph, g.first, g.count, (long)first, (long)count);
            return 1;
          }
          ++checked;
        }
      }
    }
  std::printf("%ld checked\n", checked);
  return checked > 1000 ? 0 : 2;
}
"""


def test_groups_of_a_phase(tmp_path):
    src, exe = tmp_path / "groups.cpp", tmp_path / "groups"
    src.write_text(PROGRAM)
    inc = os.path.join(ROOT, "nvfp4_w4a16_lm_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-I", inc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
