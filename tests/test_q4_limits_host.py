"""The limits and the held size that the header states for 4-bit weights are those of the code."""
import ctypes
import os
import re

import pytest

from decode_gemv_sign_gb300 import wcomp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from decode_gemv_sign_gb300 import build

    build.build()
    return wcomp.lib()


@pytest.fixture(scope="module")
def header():
    with open(os.path.join(ROOT, "include", "wcomp.h")) as f:
        return re.sub(r"\s+\*?\s*", " ", f.read())  # on one line, without the asterisks of comments and products


def test_the_stated_limit_on_rows(lib, header):
    rows = int(re.search(r"M ceil\(N / (\d+)\) below 2\^31", header).group(1))
    h, x = ctypes.c_void_p(), ctypes.c_void_p(256)
    per = 1 << 15  # row tiles a matrix: 2^16 matrices reach the limit
    for N, refused in ((per * rows, True), ((per - 1) * rows + 1, True), ((per - 1) * rows, False)):
        # what is within the limits ends at the device: none here, or no memory for it
        st = lib.wcomp_q4_encode(x, 1 << 16, N, 1 << 20, 32, None, ctypes.byref(h))
        assert (st == wcomp.EUNSUPPORTED) == refused and st != wcomp.OK and not h.value, (N, st)


def test_the_stated_size_is_that_of_the_layout(header):
    m = re.search(r"M ceil\(N / (\d+)\) ceil\(K / (\d+)\) blocks of (\d+) rows x (\d+) columns, each (\d+) bytes of "
                  r"codes and (\d+) / group bytes of scales", header)
    rows, cols, rows2, cols2, codes, scales = map(int, m.groups())
    with open(os.path.join(ROOT, "decode_gemv_sign_gb300", "csrc", "tile.cuh")) as f:
        src = f.read()

    def constant(name):
        return int(re.search(rf"constexpr int {name} = (\d+)", src).group(1))

    assert rows == rows2 == constant("kTileRows") and cols == cols2 == constant("kQ4Cols")
    assert codes == rows * cols // 2 and scales == rows * cols * 2
