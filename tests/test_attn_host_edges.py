"""CPU checks of the attention operators at the ends of their ranges."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int4_w4a16_group_gb300", "csrc")

BORDERS = r"""
#include <cstdio>
#include <initializer_list>
#include <limits.h>
#include "kv_layout.h"
using namespace w4a16;
int main() {
  const int tokens = 1 << 30;          // the most a block table may hold
  for (int len : {0, 1, 3, 120, tokens})
    for (int n : {1, 2, 40, 300, INT_MAX / 8})
      for (int window : {1, 2, 16, 1 << 30, INT_MAX - 300, INT_MAX - 1, INT_MAX})
        for (int i : {0, 1, 2, 37, 39, n - 1}) {
          if (i >= n) continue;
          bool bad = false;
          const KvSeq s = kv_sequence(0, n, len, INT_MAX, tokens, &bad);
          if (bad) return 1;
          const long long pos = (long long)len - n + i;
          const long long lo = pos + 1 - window, hi = pos + 1;
          if (kv_lo(s, i, window) != (lo < 0 ? 0 : lo)) return 2;
          if (kv_lo(s, i, 0) != 0) return 3;
          if (kv_hi(s, i, 1, false) != (hi < 0 ? 0 : hi)) return 4;
        }
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_borders_of_any_window(tmp_path):
    """Windows up to the largest int, query tokens before the first key among them, without signed overflow."""
    src, exe = tmp_path / "borders.cpp", tmp_path / "borders"
    src.write_text(BORDERS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
