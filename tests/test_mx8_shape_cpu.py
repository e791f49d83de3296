"""The choice between chunks of a few rows and tiles for up to 16 rows of 8 bits and a long K, without a GPU (csrc/mx_shape.h
is plain C++)."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_mixture_experts_moe_amd", "csrc")
CUS = 256

PROGRAM = """
#include "mx_shape.h"
#include <stdio.h>
int main() {
  long long n, chunks; int whole, cus;
  while (scanf("%lld %lld %d %d", &n, &chunks, &whole, &cus) == 4) printf("%d\\n", (int)k3moe::mx8_few_in_chunks((int)n, chunks, whole != 0, cus));
}
"""

# N, K, chunks; us in chunks, in tiles, as measured on 256 CUs
MEASURED = [(300, 9216, 2, 7.9, 7.8), (2048, 9216, 2, 8.5, 11.7), (4096, 9216, 2, 15.7, 15.2), (7168, 9216, 2, 22.9, 15.4), (33792, 9216, 2, 73.0, 47.0),
            (1024, 12288, 2, 9.4, 8.6), (4096, 12288, 2, 17.6, 19.0), (7168, 12288, 2, 27.1, 22.9), (16384, 12288, 2, 45.9, 27.0),
            (2048, 16384, 2, 11.6, 24.1), (4096, 16384, 2, 22.3, 24.1), (7168, 16384, 2, 32.8, 30.1), (33792, 16384, 2, 112.0, 80.7),
            (2048, 24576, 4, 24.7, 33.9), (4096, 24576, 3, 38.5, 41.7), (4096, 24576, 4, 50.1, 42.1), (7168, 24576, 4, 78.4, 44.1),
            (2048, 33792, 4, 31.4, 45.3), (4096, 33792, 3, 51.2, 55.8), (4096, 33792, 4, 66.8, 56.7), (7168, 33792, 2, 54.6, 55.8),
            (7168, 33792, 3, 78.6, 56.9), (7168, 33792, 4, 103.0, 58.0), (33792, 33792, 4, 448.2, 161.8),
            (1024, 65536, 8, 48.1, 83.9), (2048, 65536, 6, 76.0, 101.0), (2048, 65536, 8, 100.6, 102.5), (4096, 65536, 4, 123.9, 102.5),
            (16384, 65536, 8, 947.2, 131.7),
            (2048, 9248, 2, 9.4, 12.9), (4096, 9248, 2, 17.6, 22.1), (7168, 9248, 2, 24.7, 23.1), (9000, 9248, 2, 31.9, 29.6), (16384, 9248, 2, 42.8, 33.0),
            (4096, 16416, 2, 24.7, 36.0), (9000, 16416, 2, 49.6, 52.2), (16384, 16416, 2, 64.8, 54.9),
            (7168, 33760, 2, 63.3, 96.6), (7168, 33760, 3, 91.5, 98.0), (5500, 33760, 4, 91.5, 101.9), (7168, 33760, 4, 120.1, 99.0), (16384, 33760, 4, 247.6, 109.1),
            (4096, 65568, 4, 116.5, 188.3), (4096, 65568, 6, 169.2, 190.2), (4096, 65568, 8, 222.0, 189.5), (16384, 65568, 8, 900.1, 209.2),
            (1024, 100000, 16, 150.7, 279.3), (2048, 100000, 12, 226.5, 279.6), (4096, 100000, 5, 203.5, 275.3), (4096, 100000, 12, 468.6, 282.0),
            (7168, 100000, 2, 171.7, 276.2), (7168, 100000, 16, 1168.4, 289.4)]


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++") or shutil.which("clang++") or "/opt/rocm/bin/amdclang++"
    d = tmp_path_factory.mktemp("mx8_shape")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(d / "p.cpp"), "-o", str(d / "p")], check=True)

    def ask(lines):
        text = "\n".join(" ".join(str(int(v)) for v in line) for line in lines) + "\n"
        return [line == "1" for line in subprocess.run([str(d / "p")], input=text, capture_output=True, text=True, check=True).stdout.split()]

    return ask


def test_the_choice_is_not_the_slower_one(choose):
    for (n, k, chunks, few, tiles), taken in zip(MEASURED, choose([(n, c, k % 512 == 0, CUS) for n, k, c, _, _ in MEASURED])):
        assert (few if taken else tiles) <= 1.1 * min(few, tiles), (n, k, chunks)


def test_one_chunk_always_and_the_largest_sizes(choose):
    most = 2**31 - 1
    assert choose([(most, 1, True, CUS), (1, 1, False, 1), (most, 2, True, CUS), (most, 16, False, 4096), (1, 16, True, CUS)]) == [True, True, False, False, True]
