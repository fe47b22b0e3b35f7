"""The norms' plans (csrc/la2_norm_plan.h) and the answers kept about a device
(csrc/la2_memo.h), built as host programs: which CTA and thread takes which
columns, over every width; which questions are asked again."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

GATED = r"""
#include <cstdio>
#include <cstring>
#include "la2_norm_plan.h"
using namespace la2::norm_plan;
// The units of the CTAs that share a row (or, per head, a slice's) as the
// kernel places them: every column once, no unit across a head's end.
static bool covered(const NormPlan &g, int D, int e, int bytes) {
  static char seen[1 << 16];
  std::memset(seen, 0, sizeof seen);
  for (int part = 0; part < g.cl * g.slices; part++) {
    const int c0 = part * g.cols, end = c0 + g.cols < D ? c0 + g.cols : D;
    for (int u = 0; u < g.nv * g.tpr; u++) {
      const int c = c0 + gated_unit(bytes, u);
      if (c >= end) continue;
      const int last = c + gated_apart(bytes);
      if (c / e != (last + 3) / e) return false;
      for (int i = 0; i < 4; i++) seen[c + i]++, seen[last + i]++;
    }
  }
  for (int c = 0; c < (1 << 16); c++)
    if (seen[c] != (c < D)) return false;
  return true;
}
int main() {
  for (int e = 64; e <= 128; e += 64)
    for (int H = 1; H * e <= kNormMaxCols; H++)
      for (int bytes = 2; bytes <= 4; bytes += 2) {
        if (!covered(gated_row_plan(H * e, bytes), H * e, e, bytes)) std::printf("row %d %d %d\n", H, e, bytes);
        if (!covered(head_plan(H, e), H * e, e, bytes)) std::printf("head %d %d %d\n", H, e, bytes);
      }
}
"""


def run(tmp_path, source):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(source)
    include = os.path.join(ROOT, "causal_linear_attention_fwd_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", include, "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout


def test_gated_rows_are_covered_once(tmp_path):
    """Every head count and size up to the widest row, 16 and 32 bits."""
    assert run(tmp_path, GATED) == ""


MEMO = r"""
#include <cstdio>
#include "la2_memo.h"
static int asked = 0;
static int get(la2::DeviceMemo &m, int dev, uint64_t key, bool works, int answer) {
  return m.get(dev, key, 1, [&](int *n) { asked++; *n = answer; return works; });
}
int main() {
  static la2::DeviceMemo m;
  int bad = 0;
  auto expect = [&](int got, int want, int questions) {
    if (got != want || asked != questions) std::printf("%d: %d %d, %d questions\n", ++bad, got, want, asked);
  };
  expect(get(m, 0, 100, false, 9), 1, 1);    // failed: the stand-in, and not kept
  expect(get(m, 0, 100, true, 4), 4, 2);
  expect(get(m, 0, 100, true, 7), 4, 2);     // kept
  expect(get(m, 1, 100, true, 3), 3, 3);     // another device has its own
  expect(get(m, 0, 100, true, 7), 4, 3);
  expect(get(m, 0, 200, true, 2), 2, 4);     // another size
  expect(get(m, 1, 100, true, 7), 3, 4);
  expect(get(m, 0, 0, true, 5), 5, 5);       // no shared memory is a size too
  expect(get(m, 0, 0, true, 7), 5, 5);
  expect(get(m, 64, 100, true, 6), 6, 6);    // past the devices that are kept, or none
  expect(get(m, -1, 100, true, 6), 6, 7);
  expect(get(m, 2, 100, true, 0), 1, 8);     // no CTA fits: the stand-in
}
"""


def test_answers_are_kept_by_device(tmp_path):
    assert run(tmp_path, MEMO) == ""


RESIDUAL = r"""
#include <cstdio>
#include "la2_norm_plan.h"
using namespace la2::norm_plan;
static_assert(most_cl(false) >= 1 && most_cl(true) >= 1, "known to the compiler");
int main() {
  for (int D = 1; D <= kNormMaxCols; D++)
    for (int odd = 0; odd <= (D % 8 != 0); odd++) {
      if (D % 8 != 0 && !odd) continue;
      for (int units = 2; units <= (odd ? 2 : 4); units += 2) {
        const NormPlan g = row_plan(D, odd, units);
        const int places = odd ? D + 7 : D;
        // every place has a thread, every CTA a column, and the arrays of
        // partial sums room for the cluster
        const bool ok = g.cols % 8 == 0 && g.cl * g.cols >= places && (g.cl - 1) * g.cols < D &&
                        g.tpr * g.nv * 8 >= g.cols && g.nt == g.tpr * g.rpc && g.cl <= most_cl(odd) &&
                        (g.cl == 1 || g.rpc == 1);
        if (!ok) std::printf("%d %d %d\n", D, odd, units);
      }
    }
}
"""


def test_rows_have_threads_and_room(tmp_path):
    """Every width, the forward's four units and the backward's two."""
    assert run(tmp_path, RESIDUAL) == ""
