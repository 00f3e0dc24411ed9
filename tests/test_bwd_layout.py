"""Where the backward kernels keep P^T in tensor memory, checked on the host:
the two warps of a lane quarter are not ordered between the arrival of S^T and
the product that reads P^T, so neither may store over scores of the other."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_99_gb300", "csrc")
KERNELS = ["fa_bwd.cu", "fa_seq_bwd.cu"]

PROGRAM = r"""
#include "fa_bwd_layout.h"
#include <cstdio>
int main() {
  int bad = 0;
  // a warp's 64 query rows as bf16 pairs: 32 columns, all of which it read itself
  for (int c0 = 0; c0 < 128; c0 += 64)
    for (int c = 0; c < 32; ++c) {
      const int col = fa::p_store_col(c0) + c;
      if (col < c0 || col >= c0 + 64) ++bad;
    }
  // the product finds query row r where its warp put it
  for (int r = 0; r < 128; ++r)
    if (fa::p_operand_col(r / 16) + r % 16 / 2 != fa::p_store_col(r / 64 * 64) + r % 64 / 2) ++bad;
  std::printf("%d\n", bad);
}
"""


def test_a_warp_stores_over_its_own_scores(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.strip() == "0"


@pytest.mark.parametrize("name", KERNELS)
def test_the_kernels_use_that_layout(name):
    text = open(os.path.join(CSRC, name)).read()
    assert "kColS + p_store_col(c0) + c * 16" in text and "tmem + C::kColS + p_operand_col(kk)" in text
