"""The rule by which blocks of 16 and 32 rows are streamed or taken by tiles, in the host's code: on
both sides of the loads where either was measured to be the faster."""
import os
import subprocess

import pytest

from moe_expert_layer_segment_amd import build

PROGRAM = r"""
#include <cstdio>
#include "kernels.hpp"
int main() {
  const int blocks[] = {16, 32, 48}, loads[] = {4, 8, 12, 16, 20, 24, 32, 64};
  const int32_t ids = 0;
  for (int bm : blocks)
    for (int per : loads)
      for (int with_ids = 0; with_ids < 2; ++with_ids) {
        moelora::Int8Gemm p = {};
        p.E = 32;
        p.BM = bm;
        p.num_ids = 32 * per;
        p.row_ids = with_ids ? &ids : nullptr;
        p.M = 32 * per + 32 * bm / 2;   // blocks whose last are half full
        printf("%d %d %d\n", bm, per, (int)moelora::int8_few_rows(p));
      }
}
"""


@pytest.mark.skipif(not os.path.exists(build.hipcc()), reason="hipcc missing")
def test_blocks_are_streamed_where_that_is_faster(tmp_path):
    src, exe = tmp_path / "rule.hip", tmp_path / "rule"
    src.write_text(PROGRAM)
    subprocess.run([build.hipcc(), *build.common_flags(), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    got = {}
    for line in filter(None, out):
        bm, per, few = map(int, line.split())
        got.setdefault((bm, per), set()).add(few)
    assert got == {(bm, per): {int(per <= {16: 12, 32: 20, 48: 0}[bm])} for bm in (16, 32, 48)
                   for per in (4, 8, 12, 16, 20, 24, 32, 64)}
