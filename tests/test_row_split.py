"""How a row of logits is shared out over a cluster (csrc/row_split.h), compiled for the host: every block and every group of
words belongs to exactly one CTA, and a CTA's groups begin in blocks of its own. A group of two CTAs would be two
unordered writes of one maximum."""
import os
import subprocess

from hybrid_upcycling_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "row_split.h"
using namespace hylo;
int main() {
  long cases = 0, empty = 0;
  for (int vec = 4; vec <= 8; vec *= 2)  // words of a 16-byte vector: fp32, 16 bits
    for (long v = 1; v < 40000000; v = v < 3000 ? v + 1 : v < 400000 ? v + 61 : v + v / 37 + 1)
      for (int lead = 0; lead < vec; lead += vec - 1) {
        const long host = (v + vec - 1 + 32 * vec - 1) / (32 * vec);  // blocks wherever the row starts
        const int blocks = (int)((v + lead + 32 * vec - 1) / (32 * vec));
        int shift = 0;
        while (((host * 32 + (1L << shift) - 1) >> shift) > 256) ++shift;
        const int per = shift < 5 ? 5 - shift : 0, down = shift > 5 ? shift - 5 : 0;
        const int groups = ((blocks << per) + (1 << down) - 1) >> down;
        for (int ctas = 1; ctas <= 16; ctas *= 2) {
          const int span = row_span(host, ctas, shift);
          std::vector<int> owner(groups, -1);
          int next = 0;
          for (int q = 0; q < ctas; ++q) {
            const RowPart r = row_part(blocks, span, q, shift);
            bool bad = r.blk0 != next || r.blk1 < r.blk0 || r.blk1 > blocks || span % 4 != 0;
            next = r.blk1;
            for (int g = r.g0; g < r.g1; ++g) {
              const int first = (g << down) >> per;  // the group's first block
              bad = bad || g >= groups || owner[g] >= 0 || first < r.blk0 || first >= r.blk1;
              if (g < groups) owner[g] = q;
            }
            if (bad) return printf("V=%ld vec=%d lead=%d ctas=%d: CTA %d\n", v, vec, lead, ctas, q), 1;
            empty += r.blk0 == r.blk1;
          }
          for (int g = 0; g < groups; ++g)
            if (owner[g] < 0) return printf("V=%ld vec=%d lead=%d ctas=%d: group %d of nobody\n", v, vec, lead, ctas, g), 1;
          if (next != blocks || groups > 256) return printf("V=%ld vec=%d ctas=%d: blocks\n", v, vec, ctas), 1;
          ++cases;
        }
      }
  printf("%ld cases, %ld CTAs without blocks\n", cases, empty);
  return empty > 0 ? 0 : 1;
}
"""


def test_blocks_and_groups_have_one_owner(tmp_path):
    src, exe = tmp_path / "row_split.cpp", tmp_path / "row_split"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(build.CSRC), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
