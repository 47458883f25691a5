"""The record of which kernels have had their shared-memory limit raised
(csrc/smem_table.h): a process that uses every kernel of the library on
several GPUs stays within it, so no call sets the attribute twice.  Compiled
here on its own; no GPU needed."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_gemm_b200", "csrc")

PROGRAM = r"""
#include "smem_table.h"
#include <cstdio>
using svdq::SmemTable;
static SmemTable t;
static char kernels[300];

int main() {
  // 300 kernels (the library has fewer than 250) on 8 devices, each asked for twice
  int sets = 0;
  for (int round = 0; round < 2; ++round)
    for (int dev = 0; dev < 8; ++dev)
      for (int k = 0; k < 300; ++k)
        if (t.raised(&kernels[k], dev) < 1000 + (size_t)k) {
          ++sets;
          t.note(&kernels[k], dev, 1000 + k);
        }
  if (sets != 8 * 300) return printf("%d limits set for 2400 kernels\n", sets), 1;
  // one (kernel, device) is not another
  if (t.raised(&kernels[3], 9) != 0 || t.raised(&kernels[3], 1) != 1003) return printf("mixed up\n"), 1;
  // a limit only grows
  t.note(&kernels[3], 1, 5000);
  if (t.raised(&kernels[3], 1) != 5000) return printf("not grown\n"), 1;
  // more than it holds: it forgets the new ones, keeps the old ones and ends every search
  static char many[2 * SmemTable::SIZE];
  for (char& c : many) t.note(&c, 0, 7);
  for (int k = 0; k < 300; ++k)
    if (t.raised(&kernels[k], 7) != 1000 + (size_t)k) return printf("lost an entry\n"), 1;
  int known = 0;
  for (char& c : many) known += t.raised(&c, 0) == 7;
  if (known != SmemTable::SIZE / 4 * 3 - 2400) return printf("%d known\n", known), 1;
  puts("ok");
  return 0;
}
"""


def test_smem_table(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "t.cc", str(tmp_path / "t")
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, "-o", exe, str(src)], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.stdout == "ok\n", r.stdout
