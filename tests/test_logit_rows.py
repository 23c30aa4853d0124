"""Which 16-byte blocks of a row of logits fp4_logprobs and its gradient load
whole (CPU: csrc/logit_rows.h, which the kernels compile too): those, and all
of those, that lie within the matrix."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "block_scaled_fp4_03_amd", "csrc")


@pytest.fixture(scope="module")
def blocks(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rows") / "logit_rows_check.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(HERE, "logit_rows_check.cpp"), "-o", so], check=True)
    f = ctypes.CDLL(so).logit_row_blocks
    f.argtypes = [ctypes.c_uint32, ctypes.c_uint64] + [ctypes.c_uint32] * 4 + [ctypes.c_void_p]
    f.restype = None

    def run(size, at, n, rows, stride, V):
        out = (ctypes.c_uint32 * 4)()
        f(size, at, n, rows, stride, V, out)
        return tuple(out)

    return run


@pytest.mark.parametrize("size", (2, 4))
@pytest.mark.parametrize("V", (1, 2, 3, 5, 7, 8, 9, 15, 31, 64, 65, 200))
def test_whole_blocks_lie_within_the_matrix(blocks, size, V):
    start = 1 << 20
    for gap in (0, 1, 3, 70):
        stride = V + gap
        for rows in (1, 2, 3, 5, 12, 70):
            for shift in sorted({0, size, 16 - size, 16, 48, 128 - size}):
                first = start + shift
                end = first + ((rows - 1) * stride + V) * size
                for n in range(rows):
                    at = first + n * stride * size
                    head, count, lo, hi = blocks(size, at, n, rows, stride, V)
                    what = "size %d V %d stride %d row %d of %d at +%d" % (size, V, stride, n, rows, shift)
                    line = at - head * size
                    assert line % 128 == 0 and at - line < 128, what
                    assert line + 16 * count >= at + V * size > line + 16 * (count - 1), what
                    whole = [j for j in range(count) if line + 16 * j >= first and line + 16 * j + 16 <= end]
                    assert list(range(lo, hi)) == whole or (lo >= hi and not whole), what


def test_of_the_largest_rows(blocks):
    """Counts near 2^31 elements do not wrap."""
    V = (1 << 31) - 1
    for size in (2, 4):
        E = 16 // size
        head, count, lo, hi = blocks(size, 128 - size, 0, 1, V, V)
        assert head == 128 // size - 1 and count == (V + head + E - 1) // E
        assert lo == (head + E - 1) // E and hi == (count - 1 if count * E > head + V else count)
