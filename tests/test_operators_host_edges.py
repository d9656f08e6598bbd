"""Host checks of the 4-bit and cache operators that need no device: the rule by which CTAs share a tile, and what
a stream given by hand holds on to."""
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


class FakeTensor:
    is_cuda = True

    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


class FakeStream:
    """Stands for a torch stream, or with `device` for one made around a handle."""

    def __init__(self, handle, device=None):
        self.cuda_stream = handle


def test_stream_handle_is_not_kept(monkeypatch):
    """A torch stream holds on to a call's tensors; one given as its handle is never handed to the allocator, which
    would use it when they are freed, and the default stream's, 0, is torch's own."""
    import contextlib

    import torch

    from dit_weight_compression_b200 import operators
    default = FakeStream(0)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", type("Outside", (FakeStream,), {}))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d: default)
    dev, x, s = torch.device("cuda", 0), FakeTensor(), FakeStream(77)
    assert operators._on(dev, s, x, None)[1] == 77 and x.streams == [s]
    x.streams.clear()
    for given in (78, torch.cuda.ExternalStream(78)):
        assert operators._on(dev, given, x, None)[1] == 78 and x.streams == []
    assert operators._on(dev, 0, x, None)[1] == 0 and x.streams == [default]
