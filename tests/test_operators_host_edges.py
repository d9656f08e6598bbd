"""Host checks of the 4-bit and cache operators that need no device: the rule by which CTAs share a tile."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dit_weight_compression_b200", "csrc")

SPLIT_PROBE = r"""
#include "fp4_shape.h"
#include <cstdio>
#include <cstdlib>
// argv: tiles, steps, then the clusters of 1, 2, ... 8 CTAs that the device holds (-1: an error)
int main(int argc, char** argv) {
    int split = 0;
    const int e = ep::fp4::split_of(atoll(argv[1]), atoi(argv[2]), [&](int n, int& clusters) {
        clusters = atoi(argv[2 + n]);
        return clusters < 0 ? 7 : 0;
    }, 9, split);
    printf("%d %d\n", e, split);
    return 0;
}
"""


@pytest.fixture(scope="module")
def split_of(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("split")
    src, exe = d / "probe.cpp", d / "probe"
    src.write_text(SPLIT_PROBE)
    subprocess.run([cxx, "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def run(tiles, steps, room):
        out = subprocess.run([str(exe), str(tiles), str(steps), *map(str, room)], check=True, capture_output=True, text=True)
        return tuple(map(int, out.stdout.split()))
    return run


WHOLE = (296, 148, 98, 74, 58, 48, 41, 36)  # a GPU of 148 SMs, two CTAs each


@pytest.mark.parametrize("tiles,steps,room,want", [
    (1, 32, WHOLE, (0, 8)), (36, 32, WHOLE, (0, 8)), (37, 32, WHOLE, (0, 7)), (224, 32, WHOLE, (0, 1)), (32, 16, WHOLE, (0, 4)),
    (1, 1, WHOLE, (0, 1)), (1, 5, WHOLE, (0, 2)), (100000, 32, WHOLE, (0, 1)),
    # a part of a GPU on which large clusters, or any, find no room
    (1, 32, (8, 4, 2, 2, 0, 0, 0, 0), (0, 4)), (2, 32, (8, 4, 2, 1, 0, 0, 0, 0), (0, 3)), (1, 32, (8, 0, 0, 0, 0, 0, 0, 0), (0, 1)),
    (9, 32, (8, 4, 2, 1, 0, 0, 0, 0), (0, 1)),
    # nothing fits, or the device does not answer
    (1, 32, (0,) * 8, (9, 1)), (1, 32, WHOLE[:7] + (-1,), (7, 8)), (1, 1, (-1,) + WHOLE[1:], (7, 1))])
def test_ctas_of_a_tile(split_of, tiles, steps, room, want):
    assert split_of(tiles, steps, room) == want
