"""Launch arithmetic of the microscaled products up to the largest sizes that
the header allows (2^31 - 1 rows or columns), without a GPU: csrc/mx_shape.h is
plain C++, so a host program prints what the launches and kernels compute."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_mixture_experts_moe_amd", "csrc")
MOST = 2**31 - 1
SIZES = [1, 15, 16, 17, 33792, 2**20 + 1] + [MOST - d for d in (0, 1, 14, 15, 16, 31, 62, 63, 64, 65, 126, 127, 128, 254, 255, 256, 1000)]
CUS = 256

PROGRAM = """
#include "mx_shape.h"
#include <stdio.h>
using namespace k3moe;
int main() {
  long long n, m; int side;
  char kind;
  while (scanf(" %c %lld %lld %d", &kind, &m, &n, &side) == 4) {
    if (kind == 'f') {
      const MxFewGrid g = mx_few_grid((int)n, side, (int)m);
      printf("%d %lld %d %d\\n", g.rounds, (long long)g.wgs, mx_few_rounds((int)n, side, (int)g.wgs), mx_groups((int)n, 16));
    } else {
      const MxTileGrid g = mx_tile_grid((int)m, (int)n, side);
      printf("%lld %u %u %d\\n", (long long)g.total, g.x, g.y, mx_groups((int)n, side));
    }
  }
}
"""


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++") or "/opt/rocm/bin/amdclang++"
    d = tmp_path_factory.mktemp("mx_shape")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(d / "p.cpp"), "-o", str(d / "p")], check=True)

    def ask(lines):
        out = subprocess.run([str(d / "p")], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
        return [[int(v) for v in line.split()] for line in out.splitlines()]

    return ask


def test_few_row_groups_and_rounds(shape):
    """Every group is reached, by as many rounds as the kernel counts, and no count is negative."""
    asked = [(n, rw) for n in SIZES for rw in range(1, 9)]
    got = shape([f"f {CUS} {n} {rw}" for n, rw in asked])
    for (n, rw), (rounds, wgs, kernel_rounds, groups) in zip(asked, got):
        want = -(-n // 16)
        assert groups == want, (n, rw)
        assert rounds == -(-want // (2 * CUS * rw)) and kernel_rounds == rounds, (n, rw, rounds, kernel_rounds)
        assert 1 <= wgs <= 2 * CUS and wgs * rw * rounds >= want > 0, (n, rw, wgs)
        assert (rounds + 3) * wgs * rw < 2**31  # group numbers that are asked for ahead


def test_tile_grids(shape):
    asked = [(m, n, s) for s in (64, 128, 256) for n in SIZES for m in (1, 17, 64, 65, 200, 257)]
    asked += [(n, m, s) for m, n, s in asked]
    got = shape([f"t {m} {n} {s}" for m, n, s in asked])
    for (m, n, s), (total, x, y, columns) in zip(asked, got):
        assert columns == -(-n // s), (m, n, s)
        assert total == -(-m // s) * -(-n // s), (m, n, s)
        assert 1 <= x <= 2**20 and 1 <= y < 65536 and (y - 1) * x < total <= x * y, (m, n, s)
