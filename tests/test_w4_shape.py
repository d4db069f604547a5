"""What the 4-bit products ask for as LDS against what their workgroups address, over sizes and rows: the
library's own functions (csrc/w4_shape.h), compiled by g++. An expert that tokens name more than once
has more rows than there are tokens; a layout for the tokens alone would be too small for them, which the last
lines hold against the sizes that such a layout had."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routing_grouped_expert_gemm_amd", "csrc")

DRIVER = r"""
#include <stdio.h>
#include "w4_shape.h"
using namespace mok;
static long bad = 0, seen = 0;
// rows: with the tokens' one route each; most: of all routes
static void one(bool few, int g, int pl, int K, long long waves, int pair, int red, long long T, long long routes) {
  const int mr = few ? 4 : pl > 1 ? 8 : 16, bodies = (K + W4_BODY - 1) / W4_BODY;
  const int rows = (int)(T < mr ? T : mr), most = (int)(routes < mr ? routes : mr);
  const W4Shape s = w4_shape(few, g, pl, K, waves, pair, red, rows, most);
  bool ok = s.ks >= 1 && s.ks <= bodies && s.tpw >= pair && s.tpw * s.ks <= W4_MAXW && s.tpw % pair == 0 &&
            s.lds + 8192 <= 160 * 1024 && s.lds >= (size_t)s.tpw * s.ks * red;
  for (int n = 1; n <= most; ++n) ok = ok && w4_x_bytes(few, g, pl, bodies, s.ks, s.cap, n) <= s.lds;
  ++seen;
  if (!ok && ++bad < 10) printf("few %d g %d planes %d K %d waves %lld T %lld routes %lld: lds %zu\n", few, g, pl, K, waves, T, routes, s.lds);
}
int main() {
  const int groups[] = {32, 64, 128};
  const long long waves[] = {1, 16, 100, 700, 1500, 2048, 100000};
  for (int g : groups)
    for (int K = g; K <= 20000; K += K < 2000 ? g : 7 * g)
      for (long long w : waves)
        for (int T = 1; T <= 20; ++T)
          for (int k = 1; k <= 16; k += k < 4 ? 1 : 6) {
            one(true, g, 1, K, w, 2, 0, T, (long long)T * k);
            one(true, g, 1, K, w, 1, 0, T, (long long)T * k);
            one(false, g, 1, K, w, 1, 2048, T, (long long)T * k);
            one(false, g, PLANES, K, w, 1, 1024, T, (long long)T * k);
          }
  for (int g : groups)
    for (int K = g; K <= 20000; K += g)
      for (int k = 1; k <= W4_MAXW; ++k) {
        const W4Shape s = w4_token_shape(g, K, k);
        ++seen;
        if (s.ks < 1 || s.ks * k > W4_MAXW || w4_x_bytes(true, g, 1, (K + W4_BODY - 1) / W4_BODY, s.ks, s.cap, k) > s.lds) ++bad;
      }
  printf("%ld %ld\n", seen, bad);
  // one token, two picks of one expert, K 512, groups of 32: a layout for one row, and what two rows address
  const W4Shape one_row = w4_shape(true, 32, 1, 512, 1 << 20, 2, 0, 1, 1), both = w4_shape(true, 32, 1, 512, 1 << 20, 2, 0, 1, 2);
  printf("%zu %zu %zu\n", one_row.lds, w4_x_bytes(true, 32, 1, 1, one_row.ks, one_row.cap, 2), both.lds);
  return 0;
}
"""


def test_requested_covers_what_is_addressed(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src = open(os.path.join(CSRC, "w4.hip")).read()
    planes = int(src.split("PL = MODE == W4_DOWN ? ")[1].split(" ")[0])
    (tmp_path / "d.cpp").write_text(DRIVER)
    exe = tmp_path / "d"
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-DPLANES=%d" % planes, "-I", CSRC, str(tmp_path / "d.cpp"), "-o", str(exe)])
    lines = subprocess.check_output([str(exe)], text=True).splitlines()
    seen, bad = map(int, lines[-2].split())
    assert seen > 10000 and bad == 0, lines[:-2]
    one_row, two_rows, both = map(int, lines[-1].split())
    assert one_row < two_rows <= both
