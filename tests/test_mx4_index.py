"""Which tile a product with 4-bit weights takes (csrc/mx4_index.h), compiled
for the host: every tile is taken by sizes that the GPU tests run, and no size
makes a number of tiles that is not what the launch needs.  CPU only."""
import os
import shutil
import subprocess

import pytest

from mx4_sizes import DENSE, RAGGED, cap_of
from test_moe_index import CSRC

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "mx4_index.h"
using namespace bsq;
int main(int c, char** v) {
  const char* names[] = {"few16x16", "few16x32", "few32x32", "t32x64", "t32x64g2", "t64x64g2", "t64x128g2", "t64x128", "t128x128", "t256x256"};
  for (int i = 1; i + 8 <= c; i += 8) {
    long long x[8];
    for (int j = 0; j < 8; ++j) x[j] = atoll(v[i + j]);
    const Mx4Size s{x[0] != 0, x[1] != 0, x[2], x[3], x[4], x[5], x[6], x[7]};
    printf("%s %lld %lld\n", names[int(mx4_tile(s))], (long long)s.rows(), (long long)s.launched(16, 16));
  }
}
"""


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx4")
    (d / "index.cpp").write_text(MAIN)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=signed-integer-overflow",
                        "-fno-sanitize-recover=all", "-I", CSRC, str(d / "index.cpp"), "-o", str(d / "index")],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-3000:]

    def ask(*sizes):
        r = subprocess.run([str(d / "index")] + [str(int(v)) for v in sizes], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        name, rows, launched = r.stdout.split()
        return name, int(rows), int(launched)
    return ask


def test_each_tile_is_taken_by_a_tested_size(tile):
    for name, (B, M, N, Ks) in DENSE.items():
        for K in Ks:
            assert tile(0, 0, M, M, B, 1, N, K)[0] == name.split()[0], (name, K)
    for name, (counts, align, N, Ks) in RAGGED.items():
        cap = cap_of(counts, align)
        for K in Ks:
            for gathers in (0, 1):
                assert tile(1, gathers, cap, cap, len(counts), 2, N, K)[0] == name, (name, K)
    assert {n.split()[0] for n in DENSE} == set(RAGGED) and len(RAGGED) == 10


def test_rows_and_tiles_at_the_largest_sizes(tile):
    # choices of few tokens count, not the rows that a plan's alignment leaves empty
    assert tile(1, 1, 8, 8 * 4 + 32 * 127, 32, 4, 4096, 2048)[1] == 32
    assert tile(1, 0, 8, 500, 4, 4, 64, 64)[1] == 500
    # nothing wraps, whatever the sizes
    for sizes in ((0, 0, 1 << 30, 1 << 30, 1, 1, 16, 1 << 24), (0, 0, 16, 16, 65535, 1, 1 << 20, 32),
                  (1, 1, 1 << 30, (1 << 31) - (1 << 16), 1024, 2 ** 31 - 1, 16, 1 << 24), (1, 0, 1, 1, 1024, 1, 1 << 30, 32),
                  (0, 0, 1, 1, 1, 1, 16, 32)):
        assert tile(*sizes)[2] >= 1
