"""The scalar offsets of the streamed weights' loads, on the CPU: the range check of a buffer load compares
a lane's offset with the size minus the scalar offset, so none may be larger than the size. The header that makes
them is compiled for the host; every load of a few stacks of weights is gone through, those past the last row, past
the last step and switched off among them.
"""
import ctypes
import os
import subprocess

import pytest

MOE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_weight_only_amd", "csrc", "moe")
SOURCE = """
#include "offset.hpp"
extern "C" int row(int on, int off, int row, int row_bytes, int bytes)
{
    return fp8w::buffer_offset(on != 0, off, row, row_bytes, bytes);
}
extern "C" int plain(int on, int off, int bytes) { return fp8w::buffer_offset(on != 0, off, bytes); }
"""
CAP = 0x70000000  # the largest size a buffer is given


@pytest.fixture(scope="module")
def offsets(tmp_path_factory):
    at = tmp_path_factory.mktemp("offsets")
    (at / "offsets.cpp").write_text(SOURCE)
    lib = at / "offsets.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", MOE, str(at / "offsets.cpp"),
                    "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


# rows in the stack, bytes of a row, bytes of a row's scales (0: none), bytes that a step takes of each
STACKS = [(1, 16, 4, 256, 16), (5, 256, 16, 256, 16), (16, 2048, 128, 256, 16), (17, 4096, 0, 256, 0), (100, 1440, 92, 256, 16),
          (33, 7168, 448, 256, 16), (500, 1 << 22, 0, 256, 0), (2000, 1 << 21, 1 << 17, 256, 16)]


@pytest.mark.parametrize("rows,row_bytes,scales,step,scale_step", STACKS)
def test_no_scalar_offset_is_past_the_buffer(offsets, rows, row_bytes, scales, step, scale_step):
    steps = (row_bytes + step - 1) // step
    for first in sorted({0, max(0, rows - 17), rows - 1, rows, rows + 16, rows + 48}):  # tiles' first rows, some behind the last
        size = min(max(0, rows - first) * row_bytes, CAP)
        ssize = min(max(0, rows - first) * scales, CAP)
        for s in {0, 1, steps - 1, steps, steps + 3}:
            for on in (0, 1):
                for row in range(0, 32, 4):
                    at = offsets.row(on, step * s, row, row_bytes, size)
                    assert 0 <= at <= size
                    if on and first + row < rows and s < steps and step * s + row * row_bytes < CAP:
                        assert at == step * s + row * row_bytes
                    if not on:
                        assert at == size
                    assert 0 <= offsets.row(on, scale_step * s, row, scales, ssize) <= ssize
                assert 0 <= offsets.plain(on, step * s, size) <= size


def test_a_load_that_is_not_on_stands_at_the_end(offsets):
    for size in (0, 1, 16, 4096, CAP):
        for row in (0, 4, 28, 60):
            assert offsets.row(0, 0, row, 1 << 22, size) == size  # not behind it, whichever row it is for
        assert offsets.plain(0, 0, size) == size and offsets.plain(1, size, size) == size
