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


@pytest.fixture(scope="module")
def lib():
    from int4_w4a16_group_gb300.build import build
    build()
    import int4_w4a16_group_gb300 as w4
    return w4.C


# ------------------------------------------------------------------------------------- overlapping heads

OVERLAP = r"""
#include <cstdio>
#include <cstdlib>
#include "heads.h"
using namespace w4a16;
int main() {
  int counts[2] = {0, 0};
  for (int D : {8, 72})
    for (int T : {1, 2, 3, 5})
      for (int H : {1, 2, 3, 4, 9})
        for (int a = -6; a <= 9; ++a)
          for (int b = -6; b <= 9; ++b)
            for (int odd : {0, -4}) {
              const long long token = a * D + odd, head = b * D / 2;
              bool apart = true;
              for (int i = 0; i < T * H; ++i)
                for (int j = 0; j < i; ++j) {
                  const long long d = (i / H - j / H) * token + (i % H - j % H) * head;
                  if (llabs(d) < D) apart = false;
                }
              if (heads_disjoint(T, H, {token, head}, D) != apart) {
                printf("T %d H %d D %d token %lld head %lld\n", T, H, D, token, head);
                return 1;
              }
              ++counts[apart];
            }
  // strides whose products pass 64 bits
  const long long big = (1ll << 62);
  if (!heads_disjoint(3, 5, {big, 128}, 128) || !heads_disjoint(3, 5, {128, big}, 128)) return 2;
  if (!heads_disjoint(3, 5, {-big, big - 128}, 128) || heads_disjoint(3, 5, {-big, big - 64}, 128)) return 3;
  return counts[0] > 100 && counts[1] > 100 ? 0 : 4;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_overlap_of_strided_heads(tmp_path):
    """Against every pair of heads, for strides of either sign and order."""
    src, exe = tmp_path / "overlap.cpp", tmp_path / "overlap"
    src.write_text("#include <initializer_list>\n" + OVERLAP)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


X, P, Y = 0x10000, 0x20000, 0x30000   # fake, aligned: the check must fail before any use


@pytest.mark.parametrize("T,token,H,head,D", [
    (4, 0, 8, 128, 128), (4, 1024, 8, 0, 128), (2, 1016, 8, 128, 128), (4, 1024, 8, 120, 128), (5, 128, 8, 512, 128),
    (4, 120, 2, 4096, 128), (5, 384, 4, 512, 128),
])
def test_rope_refuses_outputs_that_overlap(lib, T, token, H, head, D):
    for dtype in (0, 1):
        assert lib.w4a16_rope(X, H * D, D, dtype, T, H, D, P, P, 16, 8, 0, 0, Y, token, head, None) == 1


def test_cache_calls_of_too_many_tokens(lib):
    """Token counters are 32 bits wide and step past the end: 2^31 - 1 tokens (keys and values by a stride of zero)
    would wrap. Both pointers are misaligned, which is refused next: no call gets as far as a launch."""
    limit = 2 ** 31 - 1 - 2 ** 24
    for T, status in ((limit, 2), (limit + 1, 3), (2 ** 31 - 1, 3)):
        assert lib.w4a16_kv_append(X + 4, 0, 128, X + 4, 0, 128, 0, T, 8, 128, P, None, None, 0, 0, 0, Y, 4, 64, None) == status
        assert lib.w4a16_kv_read(Y, 4, 64, 8, 128, P, T, X + 4, X + 4, None) == status


def test_cache_calls_of_too_many_heads(lib):
    """A token's threads are counted in 32 bits: 2^27 heads of 64 dims came to zero, and a division by it ended the
    process. As above, calls that are taken are refused for their pointers."""
    for D in (64, 128, 256):
        limit = 65535 * 256 // (D // 4)
        for Hkv, status in ((limit, 2), (limit + 1, 3), (2 ** 33 // D, 3), (2 ** 31 - 1, 3)):
            assert lib.w4a16_kv_append(X + 4, 0, 128, X + 4, 0, 128, 0, 1, Hkv, D, P, None, None, 0, 0, 0, Y, 4, 64, None) == status
            assert lib.w4a16_kv_read(Y, 4, 64, Hkv, D, P, 1, X + 4, X + 4, None) == status
