"""Where a row's parts lie, as the kernels of attention over shared prefixes tell the one that
joins them: the marks of paged.cuh, compiled into a host program."""
import os
import subprocess

from mask_aware_sparse_gb300 import build as fmbuild

PROGRAM = r"""
#include <cstdio>
#include "paged.cuh"
using namespace fm;
int main() {
  // CTAs an SM and workers of each, for GPUs of any number of SMs: whole CTAs, none too large for a mark
  for (int sms = 1; sms <= 3000; ++sms)
    for (int per_sm = 1; per_sm <= 3; ++per_sm)
      for (int warps = 1; warps <= 8; warps *= 2) {
        const int n = marked_workers(sms * per_sm, warps);
        if (n <= 0 || n % warps || n > sms * per_sm * warps || n > kMarkCtas) return printf("%d workers\n", n), 1;
        if (n < sms * per_sm * warps && n + warps <= kMarkCtas) return printf("only %d workers\n", n), 1;
        // the last worker but one and the last, and one unit that all of them share
        const int firsts[] = {0, n > 1 ? n - 2 : 0}, parts[] = {n, n > 1 ? 2 : 1};
        for (int i = 0; i < 2; ++i)
          for (int row = 0; row < kMarkRows; row += 51) {
            const uint32_t w = mark_of(firsts[i], parts[i]) | (uint32_t)row;
            if (w == kMarkWhole || mark_first(w) != firsts[i] || mark_parts(w) != parts[i] || mark_row(w) != row)
              return printf("mark %08x of %d %d %d\n", w, firsts[i], parts[i], row), 1;
          }
      }
  return marked_workers(152 * 3, 4) == 1824 ? 0 : 1;
}
"""


def test_marks_name_every_worker_and_row(tmp_path):
    src, exe = tmp_path / "marks.cu", tmp_path / "marks"
    src.write_text(PROGRAM)
    cmd = [fmbuild._nvcc(), *fmbuild.ARCH, "-std=c++17", "-I" + fmbuild.CSRC, "-I" + os.path.join(fmbuild.ROOT, "include"),
           str(src), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
