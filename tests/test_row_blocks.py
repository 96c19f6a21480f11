"""Blocks of rows of a streamed product: they cover the rows, none is longer than a block may
be, and a transposed X is copied as whole 64-row blocks only where each block starts on one."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_gemm_03_gb300", "csrc")
MOST = 9728        # 38 tiles of 256 rows, the longest that are streamed, and more


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """(M, trans_x) -> (rows of a block, whether they are whole 64-row blocks)."""
    cxx = shutil.which("g++") or pytest.skip("no g++")
    where = tmp_path_factory.mktemp("row_blocks")
    src = where / "plan.cpp"
    src.write_text("""
#include <cstdio>
#include "row_blocks.h"
int main() {
  for (int M = 1; M <= %d; ++M)
    for (int t = 0; t < 2; ++t) {
      const int rows = gb300::block_rows(M, 256, t);
      std::printf("%%d %%d %%d %%d\\n", M, t, rows, gb300::block_of_64s(M, rows));
    }
}
""" % MOST)
    exe = str(where / "plan")
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    return {(m, t): (r, w) for m, t, r, w in (map(int, line.split()) for line in out.splitlines())}


@pytest.mark.parametrize("trans", [0, 1])
def test_every_block(plans, trans):
    for M in range(1, MOST + 1):
        rows, whole = plans[M, trans]
        assert 0 < rows <= min(M, 256) and (rows % 16 == 0 or rows == M)
        assert -(-M // rows) <= -(-M // 256)              # no more blocks than full ones
        if whole:
            assert M % 64 == 0 and all(r0 % 64 == 0 for r0 in range(0, M, rows))


def test_transposed_rows_in_64s_take_the_single_copy(plans):
    assert all(plans[M, 1][1] for M in range(64, MOST + 1, 64))
